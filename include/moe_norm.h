/*
 * moe_norm.h -- C ABI of the norms before and after the expert layer, fused
 * with its gate and residual scale, and their gradients, for GB300 (sm_103a).
 *
 * The layer of moe_mxq.h maps rows x to y = layer(x).  In a block it sits
 * between two norms, and its answer enters a residual stream:
 *
 *   u = b * rsqrt(mean(b^2) + eps) * (weight_offset + w_post)     (w_post NULL: u = b)
 *   y = residual_scale * x + g * u             g = gate, or 1 / (1 + exp(-gate))
 *   n = y * rsqrt(mean(y^2) + eps) * (weight_offset + w_pre)      (w_pre NULL: no n)
 *
 * x: the stream before the layer, b: the layer's output, y: the stream after
 * it, n: the next layer's input.  One pass reads x and b once and writes y and
 * n once.  Without b (NULL) it is the first norm alone: the stream is x as it
 * is (no scale), and n its norm.
 *
 * Conventions are those of moe_mxq.h: device pointers owned by the caller, no
 * allocation, no synchronisation, work enqueued on `stream`, a moe_status
 * returned (nothing enqueued when the host detects an error).
 *   - T >= 0 rows (T = 0: a no-op; gradients of the weights are then zero);
 *     H a multiple of 8, 8 <= H <= 16384.
 *   - x, y and their gradients are of x_dtype; b, n and theirs BF16; the
 *     weights of w_dtype; the gate and its gradient of gate_dtype
 *     (enum moe_dtype).  Means, norms and sums are held in float32, and each
 *     output is rounded once: n is the norm of y before its rounding.
 *   - Row strides ldx, ldb, ldy, ldn, ld_gate in elements: multiples of 8, at
 *     least H.  Every row tensor, weight, channel gate and gradient of a weight
 *     is 16-byte aligned, a token gate and the gradients of token and channel
 *     gates as their elements (MOE_ERR_MISALIGNED).  y may be x, n may be b (each row is read before
 *     it is written); no other overlap.
 *   - gate_kind: MOE_GATE_TOKEN gate [T], MOE_GATE_CHANNEL gate [H],
 *     MOE_GATE_FULL gate [T][H] (row stride ld_gate).
 *   - Results do not depend on thread timing.
 *   - Device-side waits give up after ~1 s: the status is then MOE_ERR_TIMEOUT,
 *     what was not computed is NaN in y and n (in n the whole row), and gradients
 *     are undefined.  The debug hook of moe_get_device_status works here too.
 */
#ifndef MOE_NORM_H
#define MOE_NORM_H

#include "moe_grouped.h"

#ifdef __cplusplus
extern "C" {
#endif

enum moe_gate_kind { MOE_GATE_NONE = 0, MOE_GATE_TOKEN = 1, MOE_GATE_CHANNEL = 2, MOE_GATE_FULL = 3 };

typedef struct moe_norm_args {
    uint32_t struct_size;      /* sizeof(moe_norm_args) */
    int32_t x_dtype, w_dtype, gate_dtype;   /* enum moe_dtype */
    int32_t gate_kind;         /* enum moe_gate_kind */
    int32_t gate_sigmoid;      /* 1: g = 1 / (1 + exp(-gate)); 0: g = gate */
    float residual_scale, weight_offset, eps;
    int64_t T, H;
    const void *x;             /* [T][H]; backward: the stream y (without b: x) */
    int64_t ldx;
    const uint16_t *b;         /* [T][H] or NULL */
    int64_t ldb;
    const void *gate;          /* NULL with MOE_GATE_NONE */
    int64_t ld_gate;           /* MOE_GATE_FULL */
    const void *w_post;        /* [H] or NULL */
    const void *w_pre;         /* [H] or NULL */
    void *y;                   /* out [T][H]; NULL: not written (without b it is not) */
    int64_t ldy;
    uint16_t *n;               /* out [T][H]; NULL exactly when w_pre is */
    int64_t ldn;
    int32_t *status;           /* forward: 64 bytes of device memory, 4-byte aligned, for its device status
                                  (moe_get_device_status, reset by the call), or NULL; backward has its workspace's */
} moe_norm_args;

/* y and n as above.  residual_scale, weight_offset and eps are used as given
 * (eps >= 0). */
MOE_API int moe_norm_forward(const moe_norm_args *args, cudaStream_t stream);

typedef struct moe_norm_grads {
    uint32_t struct_size;      /* sizeof(moe_norm_grads) */
    const void *dy;            /* [T][H] x_dtype: gradient of y; NULL: zero */
    int64_t ld_dy;
    const uint16_t *dn;        /* [T][H]: gradient of n; NULL exactly when w_pre is */
    int64_t ld_dn;
    /* outputs, each NULL when not wanted */
    void *dx;                  /* [T][H] x_dtype */
    int64_t ld_dx;
    uint16_t *db;              /* [T][H] */
    int64_t ld_db;
    void *dgate;               /* as the gate: [T], [H] or [T][H] with row stride ld_dgate, gate_dtype */
    int64_t ld_dgate;
    float *dw_post;            /* [H] float32 */
    float *dw_pre;             /* [H] float32 */
    void *workspace;           /* moe_norm_workspace_size bytes, 256-byte aligned: device status (moe_get_device_status,
                                  reset by the call), sums of parts of the rows */
    size_t workspace_bytes;
} moe_norm_grads;

MOE_API size_t moe_norm_workspace_size(int64_t T, int64_t H);

/* The gradients of moe_norm_forward from those of y and n.  args are the
 * forward's with x replaced by its y (without b: x itself); y and n of args
 * are not used.  With d the whole gradient of y,
 *   d  = dy + r (dn w - h mean(dn w h)),  h = y r,  r = rsqrt(mean(y^2) + eps),  w = weight_offset + w_pre
 *   dx = residual_scale d  (without b: d)      dw_pre = sum_t dn h
 *   dgate = d u, summed over the gate's broadcast axis (times g (1 - g) with the sigmoid)
 *   db = the same norm gradient of b from g d  dw_post = sum_t g d b rsqrt(mean(b^2) + eps)
 * dx may be dy, db may be dn or b.  dw_pre needs w_pre, dw_post w_post, db b,
 * dgate a gate (MOE_ERR_INVALID_ARG). */
MOE_API int moe_norm_backward(const moe_norm_args *args, const moe_norm_grads *grads, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_NORM_H */
