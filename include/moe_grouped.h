/*
 * moe_grouped.h -- C ABI of the BF16 products grouped by expert, and their
 * gradients, for GB300 (sm_103a).
 *
 * The expert layer of moe_mxq.h runs on weights that were cast from BF16;
 * these are the products that train those BF16 weights, on the rows and the
 * offsets that moe_permute lays out.  Expert e owns rows
 * [offsets[e], offsets[e+1]) of every row tensor:
 *
 *   moe_grouped_forward:  y[r][n]     = sum_k x[r][k]  * w[e][n][k]     (r of expert e)
 *   moe_grouped_dgrad:    dx[r][k]    = sum_n dy[r][n] * w[e][n][k]     (r of expert e)
 *   moe_grouped_wgrad:    dw[e][n][k] = sum_{r of expert e} dy[r][n] * x[r][k]
 *
 * Conventions are those of moe_mxq.h: device pointers owned by the caller, no
 * allocation, no synchronisation, work enqueued on `stream`, a moe_status
 * returned (nothing enqueued when the host detects an error), device status in
 * the first bytes of the workspace (moe_get_device_status), reset by each call.
 *
 *   - Operands are BF16 (uint16_t bit patterns); sums are held in float32;
 *     outputs are rounded once to BF16, or stored as float32 (dw only).  The
 *     tensor core truncates as it adds, in norm 1e-9 of a sum for each of its
 *     terms (up to 4.5e-9 if they have one sign): beside a BF16 output's rounding
 *     that counts from some hundred thousand terms on; a float32 dw is summed in
 *     parts of 256 rows and is within a float32 product's error (3e-7, 4e-7 if
 *     they have one sign) at any length.
 *   - P rows in all (0 <= P < 2^31), N and K multiples of 8, 1 <= E <= 1024.
 *     An expert may own any number of rows, none included.
 *   - Row tensors x, y, dx, dy have a row stride in elements (ldx, ldy: a
 *     multiple of 8, at least the row's length); w and dw are contiguous
 *     [E][N][K].  Every pointer is 16-byte aligned, the workspace 256-byte
 *     (MOE_ERR_MISALIGNED).  Outputs must not overlap inputs.
 *   - offsets [E+1] int32 on the device: non-decreasing, within [0, P].  Rows
 *     outside [offsets[0], offsets[E]) (dropped pairs) belong to no expert:
 *     they are neither read into a result nor written.  Offsets that break
 *     the rule are reported in the status word (MOE_ERR_DEVICE_INDEX) and the
 *     call then writes no output.
 *   - A row's result depends on that row and its expert's weights only, and
 *     dw[e] on expert e's rows only: infinities and NaN stay where they are.
 *   - Results do not depend on thread timing.
 *   - Device-side waits give up after ~1 s (MOE_ERR_TIMEOUT).  Two SMs sum one
 *     256 x 256 tile of dw, some 4 us for 1000 rows: an expert of more than
 *     1e8 rows can take longer than that and is to be split by the caller
 *     (accumulate = 1).
 */
#ifndef MOE_GROUPED_H
#define MOE_GROUPED_H

#include "moe_mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of tensors that may have either. */
enum moe_dtype { MOE_BF16 = 0, MOE_F32 = 1 };

/* Workspace bytes of the three products for this shape (0 for invalid sizes). */
MOE_API size_t moe_grouped_workspace_size(int64_t P, int64_t N, int64_t K, int32_t E);

/* y [P][N] = x [P][K] times the transposed w [E][N][K], by expert.  Rows of no
 * expert keep what y held. */
MOE_API int moe_grouped_forward(const uint16_t *x, int64_t ldx, const uint16_t *w, const int32_t *offsets, int64_t P,
                                int64_t N, int64_t K, int32_t E, uint16_t *y, int64_t ldy, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream);

/* dx [P][K] = dy [P][N] times w [E][N][K], by expert (the gradient of
 * moe_grouped_forward's x).  Rows of no expert keep what dx held. */
MOE_API int moe_grouped_dgrad(const uint16_t *dy, int64_t ldy, const uint16_t *w, const int32_t *offsets, int64_t P,
                              int64_t N, int64_t K, int32_t E, uint16_t *dx, int64_t ldx, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/* dw [E][N][K] = transposed dy [P][N] times x [P][K] over each expert's rows
 * (the gradient of moe_grouped_forward's w), of type dw_dtype (enum moe_dtype).
 * accumulate = 0: dw is overwritten (an expert without rows gets zeros);
 * accumulate = 1: added to the float32 dw (MOE_F32 only, otherwise
 * MOE_ERR_INVALID_ARG), as gradients of micro-batches are. */
MOE_API int moe_grouped_wgrad(const uint16_t *dy, int64_t ldy, const uint16_t *x, int64_t ldx, const int32_t *offsets,
                              int64_t P, int64_t N, int64_t K, int32_t E, void *dw, int32_t dw_dtype,
                              int32_t accumulate, void *workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GROUPED_H */
