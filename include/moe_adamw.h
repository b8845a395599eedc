/*
 * moe_adamw.h -- C ABI of one AdamW step over many tensors at once, with
 * states in 32 or in 8 bits, for GB300 (sm_103a).
 *
 * For every value, with the step's number t >= 1 and g the gradient (times
 * *grad_scale when that is given, e.g. a clipping factor or 1 / loss scale):
 *
 *   m = beta1 m + (1 - beta1) g                c1 = 1 - beta1^t
 *   v = beta2 v + (1 - beta2) g^2              c2 = 1 - beta2^t
 *   p = p (1 - lr weight_decay) - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps)
 *
 * in float32 (the update to within 2^-21 of itself), p rounded once to its
 * type, and its BF16 copy (the weights that the next forward pass reads)
 * written in the same pass.
 *
 * States of 8 bits: E4M3 codes with one UE8M0 byte per 32 consecutive values,
 * the format and the rounding rule of mxq_quantize_act (moe_mxq.h).  The
 * second moment is held as its root sqrt(v), which halves the range of its
 * exponents; a root that is not zero takes at least the smallest code, so that
 * no value with a gradient ever divides by eps alone.  The step itself uses
 * the unrounded m and v.
 *
 * Conventions are those of moe_mxq.h (no allocation, no synchronisation, work
 * enqueued on `stream`, a moe_status returned; nothing is enqueued when the
 * host detects an error).  The table of tensors is read during the call and
 * may be changed or freed after it, and the numbers are part of the launch: a
 * captured one is the same step t, with the same rate and bias correction, at
 * every replay.  Each tensor is updated in place; tensors do not overlap.  A NaN
 * or an infinity stays in its value (8 bits: an infinity is held as the largest
 * value, and coarsens the other 31 of its group).
 */
#ifndef MOE_ADAMW_H
#define MOE_ADAMW_H

#include "moe_grouped.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_adamw_tensor {
    int64_t n;             /* values, >= 0 */
    void *p;               /* [n] p_dtype */
    const void *g;         /* [n] g_dtype */
    void *m, *v;           /* [n] float32; 8 bits: E4M3 codes of m and of sqrt(v) */
    uint8_t *m_scale, *v_scale;   /* 8 bits: [ceil(n / 32)] UE8M0 bytes; otherwise unused */
    uint16_t *copy;        /* [n] BF16 copy of p, or NULL (with a BF16 p: NULL) */
} moe_adamw_tensor;

typedef struct moe_adamw_args {
    uint32_t struct_size;  /* sizeof(moe_adamw_args) */
    int32_t n_tensors;
    const moe_adamw_tensor *tensors;   /* host array */
    int32_t p_dtype, g_dtype;          /* enum moe_dtype, the same for all tensors */
    int32_t state_bits;                /* 32 or 8 */
    const float *grad_scale;           /* device float, or NULL */
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;                      /* t, >= 1 */
} moe_adamw_args;

/* Every pointer is 16-byte aligned except grad_scale (4 bytes) and the scales
 * (any byte) (MOE_ERR_MISALIGNED).  0 <= beta1, beta2 < 1, eps >= 0, finite lr and
 * weight_decay, otherwise MOE_ERR_INVALID_ARG. */
MOE_API int moe_adamw_step(const moe_adamw_args *args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_ADAMW_H */
