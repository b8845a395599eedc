/*
 * moe_gated.h -- C ABI of the gated feed-forward block by expert: gate and up
 * products with their activation in one kernel, and the way back from the
 * gradient of the down product's answer to the gate and up rows, for GB300
 * (sm_103a).
 *
 * With expert e's rows r (offsets[e] <= r < offsets[e+1]), the activation f and
 * row weights v (NULL: 1):
 *
 *   moe_gated_forward:  a[r][j] = sum_k x[r][k] * w[e][j][k]      (j < 2I: gate rows, then up rows)
 *                       h[r][i] = f(a[r][i]) * a[r][I + i] * v[r]
 *   moe_gated_dgrad:    d[r][i] = sum_n dy[r][n] * w[e][n][i]     (the gradient of h)
 *                       da[r][i]     = d * v[r] * a[r][I + i] * f'(a[r][i])
 *                       da[r][I + i] = d * v[r] * f(a[r][i])
 *                       h[r][i]      = f(a[r][i]) * a[r][I + i] * v[r]   (for the down weights' gradient)
 *                       dv[r]        = sum_i d * f(a[r][i]) * a[r][I + i]
 *
 * moe_gated_forward's w is the layer's first weight, moe_gated_dgrad's its
 * second; the rest of the block are moe_grouped.h's products: the down product
 * of h, dx from da and the first weight, and both weights' gradients.
 *
 * Conventions are those of moe_grouped.h: device pointers owned by the caller,
 * no allocation, no synchronisation, work enqueued on `stream`, a moe_status
 * returned (nothing enqueued when the host detects an error), device status in
 * the first bytes of the workspace (moe_get_device_status), reset by each call.
 *
 *   - Rows, weights and outputs are BF16, v and dv float32.  Sums, activations
 *     and products are held in float32 (the tensor core truncates as it adds; for dv, where that would
 *     show, d is summed in parts: dv is off by 5e-7 in norm at H = 2048 and 1.0e-6 at 7168, by up to
 *     3.5e-6 where all terms of d have one sign); h is that of the unrounded gate and up
 *     values; every output is rounded once.  h of moe_gated_dgrad is that of the
 *     BF16 values a, as is everything else there.
 *   - 0 <= P < 2^31 rows, H and I multiples of 8, 1 <= E <= 1024 experts with any
 *     number of rows each, none included.
 *   - Row strides in elements: multiples of 8, at least the row's length.  Every
 *     pointer is 16-byte aligned, offsets, v and dv 4-byte, the workspace
 *     256-byte (MOE_ERR_MISALIGNED).  da may be a; no other overlap.
 *   - Rows of no expert are neither read into a result nor written.  Offsets that
 *     decrease or lie outside [0, P] are reported in the status word
 *     (MOE_ERR_DEVICE_INDEX), and the call then writes no output.
 *   - A row's results depend on that row, its weight and its expert's weights
 *     only: infinities and NaN stay where they are.
 *   - Results do not depend on thread timing.
 *   - Device-side waits give up after ~1 s (MOE_ERR_TIMEOUT); outputs are then
 *     undefined.
 */
#ifndef MOE_GATED_H
#define MOE_GATED_H

#include "moe_grouped.h"

#ifdef __cplusplus
extern "C" {
#endif

enum moe_activation {
    MOE_ACT_SILU = 0,          /* z / (1 + exp(-z)) */
    MOE_ACT_GELU_TANH = 1      /* z / 2 * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3))) */
};

typedef struct moe_gated_args {
    uint32_t struct_size;      /* sizeof(moe_gated_args) */
    int32_t E, activation;     /* enum moe_activation */
    int64_t P, H, I;
    const uint16_t *rows;      /* forward: x [P][H]; dgrad: dy [P][H] */
    int64_t ld_rows;
    const uint16_t *w;         /* forward: [E][2I][H]; dgrad: [E][H][I]; contiguous */
    const int32_t *offsets;    /* [E+1] */
    const float *row_w;        /* v [P] or NULL */
    uint16_t *a;               /* [P][2I]; forward: out or NULL; dgrad: in */
    int64_t ld_a;
    uint16_t *h;               /* out [P][I]; dgrad: or NULL */
    int64_t ld_h;
    uint16_t *da;              /* dgrad: out [P][2I] */
    int64_t ld_da;
    float *drow_w;             /* dgrad: out dv [P] or NULL */
    void *workspace;
    size_t workspace_bytes;
} moe_gated_args;

/* Workspace bytes of either call for this shape (0 for invalid sizes).  Each
 * call that may run at the same time as another has a workspace of its own. */
MOE_API size_t moe_gated_workspace_size(int64_t P, int64_t H, int64_t I, int32_t E);

MOE_API int moe_gated_forward(const moe_gated_args *args, cudaStream_t stream);
MOE_API int moe_gated_dgrad(const moe_gated_args *args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GATED_H */
