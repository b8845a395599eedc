/*
 * moe_muon.h -- C ABI of matrices orthogonalised by Newton-Schulz products, and
 * of a step of Muon, for GB300 (sm_103a).
 *
 * The matrices are a stack [E][N][K], e.g. the weights of E experts.  Each one,
 * for itself:
 *
 *   moe_orthogonalize:  X = x / max(|x|, eps)            (|x|: root of the sum of squares)
 *                       steps times: X = a X + (b G + c G^2) X,  G = X X^T
 *                       (over the columns, X = a X + X (b G + c G^2) with G = X^T X, where N > K)
 *                       out = X
 *   moe_muon_step:      m = mu m + (1 - mu) s g          (s: grad_scale, a device float, or 1)
 *                       u = mu m + (1 - mu) s g with nesterov, m without
 *                       p = p (1 - lr wd) - lr scale orthogonalize(u);  copy = p in BF16
 *   (K. Jordan, "Muon: An optimizer for hidden layers in neural networks", 2024)
 *
 * as AdamW's step does for the tensors that are no matrices (moe_adamw.h).
 *
 * Conventions are those of moe_mxq.h: device pointers owned by the caller, no
 * allocation, no synchronisation, work enqueued on `stream`, a moe_status
 * returned (nothing enqueued when the host detects an error); device status in
 * `status` or, where that is NULL, in the first bytes of the workspace
 * (moe_get_device_status), reset by each call.
 *
 *   - E >= 0 (0: a no-op), 1 <= N, K < 2^20, steps 0 .. 64.  All tensors are contiguous
 *     and aligned to their elements; 16-byte alignment and K a multiple of 8 are faster.
 *   - The iterates are held in FP16 with a fixed scale of 2^12, their sums in float32: eleven bits
 *     where BF16 has eight.  The polynomial enlarges what lies in directions of small singular values by up
 *     to a^steps, a rounding as well: in norm the result is off by 5e-4 to 1.2e-3 for matrices of independent
 *     values (BF16 iterates: 1e-2 to 2e-2), by up to 1.5e-2 for ones of a few large and many small singular
 *     values (0.12), by 0.05 for rank 16, 0.08 for rank 4 and 0.15 for rank 1, all of it in directions that the
 *     matrix lacks (0.4, 0.6 and 1.2; rounding such a matrix itself to BF16 costs 0.25, 0.5 and 1.15).
 *     What FP16 leaves of the diagonals of the products in between is not lost.
 *     Momentum, norm and update are computed in float32; squares that overflow float32
 *     (values of 1e18 and more) give a norm of infinity.
 *   - c is 0, or |b / (2 c)| at most 8; a, b, c at most 64 and a + b t + c t^2 at most 15.9 in magnitude for
 *     t in [0, 1] (otherwise MOE_ERR_INVALID_ARG).  The later iterates and their polynomials have to stay below 16
 *     in magnitude too, as they do for polynomials x (a + b x^2 + c x^4) that map [0, 1] into [0, 1.3].
 *   - A matrix's results depend on that matrix only: one with infinities or NaN
 *     does not change another; a matrix of zeros gives zeros.
 *   - moe_orthogonalize's out may be x if their types are the same; no other overlap.
 *   - Results do not depend on thread timing.
 *   - Device-side waits give up after ~1 s (MOE_ERR_TIMEOUT); outputs are then undefined.
 */
#ifndef MOE_MUON_H
#define MOE_MUON_H

#include "moe_grouped.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_newton_schulz {
    int32_t steps;
    float a, b, c, eps;
} moe_newton_schulz;

typedef struct moe_muon_args {
    uint32_t struct_size;      /* sizeof(moe_muon_args) */
    int32_t p_dtype, g_dtype;  /* enum moe_dtype */
    int32_t nesterov;          /* 0 or 1 */
    int64_t E, N, K;
    void *p;                   /* [E][N][K], in place */
    const void *g;
    float *m;                  /* in place */
    uint16_t *copy;            /* BF16 copy of p, or NULL */
    const float *grad_scale;   /* device float or NULL */
    double lr, momentum, weight_decay, scale;
    moe_newton_schulz ns;
    int32_t *status;           /* 64 bytes, or NULL: the workspace's */
    void *workspace;           /* 256-byte aligned */
    size_t workspace_bytes;
} moe_muon_args;

typedef struct moe_orthogonalize_args {
    uint32_t struct_size;      /* sizeof(moe_orthogonalize_args) */
    int32_t x_dtype, out_dtype;
    moe_newton_schulz ns;
    int64_t E, N, K;
    const void *x;
    void *out;
    int32_t *status;
    void *workspace;
    size_t workspace_bytes;
} moe_orthogonalize_args;

/* Workspace bytes of either call for this stack (0 for invalid sizes). */
MOE_API size_t moe_muon_workspace_size(int64_t E, int64_t N, int64_t K);

MOE_API int moe_orthogonalize(const moe_orthogonalize_args *args, cudaStream_t stream);
MOE_API int moe_muon_step(const moe_muon_args *args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_MUON_H */
