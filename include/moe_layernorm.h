/*
 * moe_layernorm.h -- C ABI of the layer norm with the residual stream's
 * addition, and its gradients, for GB300 (sm_103a).
 *
 *   s = x + b                                            (b NULL: s = x)
 *   n = (s - mean(s)) * rsqrt(var(s) + eps) * w + bias   (w NULL: 1, bias NULL: 0)
 *
 * over each row's H values, var their mean square distance from the mean.  The
 * norms of moe_norm.h have no mean and no bias.  Given dn and, of the stream
 * that goes on, ds (NULL: none), with h = (s - mean) * rsqrt(var + eps), g = dn * w:
 *
 *   dx = ds + rsqrt(var + eps) * (g - mean(g) - h * mean(g * h))     (x's and b's gradient)
 *   dw = sum over rows of dn * h,   dbias = sum over rows of dn
 *
 * Conventions are those of moe_norm.h: device pointers owned by the caller, no
 * allocation, no synchronisation, work enqueued on `stream`, a moe_status
 * returned (nothing enqueued when the host detects an error).  The kernels wait
 * for nothing, so that there is no device status.
 *   - T >= 0 rows (0: a no-op; dw and dbias are then zero); H a multiple of 8,
 *     8 <= H <= 16384.
 *   - x, s, ds, dx are of x_dtype, b, n, dn BF16, w and bias of w_dtype
 *     (enum moe_dtype), dw and dbias float32.  Means and sums are held in float32, the variance
 *     is that of the values less their mean; each output is rounded once: n is the norm of s before its rounding.
 *   - Row strides in elements: multiples of 8, at least H.  Pointers are 16-byte
 *     aligned, the workspace 256-byte (MOE_ERR_MISALIGNED).  s may be x, n may be b (without b: x),
 *     dx may be ds, s or dn, each of the same type and with the same stride; no other overlap.
 *   - A row's n, s and dx depend on that row only.
 *   - Results do not depend on thread timing.
 */
#ifndef MOE_LAYERNORM_H
#define MOE_LAYERNORM_H

#include "moe_grouped.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_layernorm_args {
    uint32_t struct_size;      /* sizeof(moe_layernorm_args) */
    int32_t x_dtype, w_dtype;
    float eps;
    int64_t T, H;
    const void *x;             /* [T][H] */
    int64_t ldx;
    const uint16_t *b;         /* [T][H] or NULL */
    int64_t ldb;
    const void *w, *bias;      /* [H] or NULL */
    void *s;                   /* out [T][H] or NULL; NULL without b */
    int64_t lds;
    uint16_t *n;               /* out [T][H] */
    int64_t ldn;
} moe_layernorm_args;

typedef struct moe_layernorm_grads {
    uint32_t struct_size;      /* sizeof(moe_layernorm_grads) */
    int32_t x_dtype, w_dtype;
    float eps;
    int64_t T, H;
    const void *s;             /* [T][H]: forward's s (without b: x) */
    int64_t lds;
    const void *w;             /* [H] or NULL */
    const uint16_t *dn;        /* [T][H] */
    int64_t ld_dn;
    const void *ds;            /* [T][H] or NULL */
    int64_t ld_ds;
    void *dx;                  /* out [T][H] or NULL */
    int64_t ld_dx;
    float *dw, *dbias;         /* out [H] or NULL; dw NULL without w */
    void *workspace;
    size_t workspace_bytes;
} moe_layernorm_grads;

/* Workspace bytes of the backward call (0 for invalid sizes).  Each call that may run at the same time as
 * another has a workspace of its own. */
MOE_API size_t moe_layernorm_workspace_size(int64_t T, int64_t H);

MOE_API int moe_layernorm_forward(const moe_layernorm_args *args, cudaStream_t stream);
MOE_API int moe_layernorm_backward(const moe_layernorm_grads *args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_LAYERNORM_H */
