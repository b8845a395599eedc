// grouped.cu -- C entry points of the BF16 products grouped by expert and their
// gradients (include/moe_grouped.h); the kernel is in grouped_kernel.cuh.
#include "grouped_kernel.cuh"

namespace mxq {

namespace {

// forward (OP kForward): in = x [P][K], out = y [P][N]; dgrad: in = dy [P][N],
// out = dx [P][K].
template <int OP>
int rows_product(const uint16_t *in, int64_t ld_in, const uint16_t *w, const int32_t *offsets, int64_t P, int64_t N,
                 int64_t K, int32_t E, uint16_t *out, int64_t ld_out, void *workspace, size_t workspace_bytes,
                 cudaStream_t st) {
  int rc = check_grouped(P, N, K, E, offsets, workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  if (P == 0)
    return cudaMemsetAsync(workspace, 0, 64, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  const int64_t R = OP == kForward ? K : N, M = OP == kForward ? N : K;
  if ((rc = check_rows(in, ld_in, R)) != MOE_OK || (rc = check_rows(out, ld_out, M)) != MOE_OK) return rc;
  if (!w) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, 16)) return MOE_ERR_MISALIGNED;
  GMaps maps;
  bool ok = OP == kForward ? encode_map(&maps.a, w, 3, K, N, E, K, N * K, GP::kBK, 128)
                           : encode_map(&maps.a, w, 3, K, N, E, K, N * K, 64, GP::kBK);
  for (int i = 0; i < 5; ++i) ok = ok && encode_map(&maps.b[i], in, 2, R, P, 1, ld_in, 0, GP::kBK, kBoxRows[i]);
  if (!ok) return MOE_ERR_CUDA;
  GArgs g{};
  g.offsets = offsets;
  g.P = P;
  g.E = E;
  g.M = (int)M;
  g.R = (int)R;
  g.ld_out = ld_out;
  g.out = out;
  g.inject_wait = injected_wait();
  g.status = reinterpret_cast<int *>(workspace);
  return launch_grouped<OP>(maps, g, most_row_items(g), st);
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" size_t moe_grouped_workspace_size(int64_t P, int64_t N, int64_t K, int32_t E) {
  if (P < 0 || N <= 0 || K <= 0 || E <= 0) return 0;
  return kStatusBytes;
}

extern "C" int moe_grouped_forward(const uint16_t *x, int64_t ldx, const uint16_t *w, const int32_t *offsets,
                                   int64_t P, int64_t N, int64_t K, int32_t E, uint16_t *y, int64_t ldy,
                                   void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return rows_product<kForward>(x, ldx, w, offsets, P, N, K, E, y, ldy, workspace, workspace_bytes, stream);
}

extern "C" int moe_grouped_dgrad(const uint16_t *dy, int64_t ldy, const uint16_t *w, const int32_t *offsets, int64_t P,
                                 int64_t N, int64_t K, int32_t E, uint16_t *dx, int64_t ldx, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  return rows_product<kDgrad>(dy, ldy, w, offsets, P, N, K, E, dx, ldx, workspace, workspace_bytes, stream);
}

extern "C" int moe_grouped_wgrad(const uint16_t *dy, int64_t ldy, const uint16_t *x, int64_t ldx,
                                 const int32_t *offsets, int64_t P, int64_t N, int64_t K, int32_t E, void *dw,
                                 int32_t dw_dtype, int32_t accumulate, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream) {
  int rc = check_grouped(P, N, K, E, offsets, workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  if ((dw_dtype != MOE_BF16 && dw_dtype != MOE_F32) || (accumulate != 0 && accumulate != 1)) return MOE_ERR_INVALID_ARG;
  if (accumulate && dw_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (!dw) return MOE_ERR_INVALID_ARG;
  if (!aligned(dw, 16)) return MOE_ERR_MISALIGNED;
  if (P == 0) {
    const size_t bytes = (size_t)E * N * K * (dw_dtype == MOE_F32 ? 4 : 2);
    if (cudaMemsetAsync(workspace, 0, 64, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return accumulate || cudaMemsetAsync(dw, 0, bytes, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  if ((rc = check_rows(dy, ldy, N)) != MOE_OK || (rc = check_rows(x, ldx, K)) != MOE_OK) return rc;
  GMaps maps;
  if (!encode_map(&maps.a, dy, 2, N, P, 1, ldy, 0, 64, GP::kBK) ||
      !encode_map(&maps.b[0], x, 2, K, P, 1, ldx, 0, 64, GP::kBK) ||
      !encode_map(&maps.b[1], dw, 3, K, N, E, K, N * K, dw_dtype == MOE_F32 ? 32 : 64, 32, dw_dtype == MOE_F32))
    return MOE_ERR_CUDA;
  GArgs g{};
  g.offsets = offsets;
  g.P = P;
  g.E = E;
  g.M = (int)N;
  g.C = (int)K;
  g.out = dw;
  g.accumulate = accumulate;
  g.inject_wait = injected_wait();
  g.status = reinterpret_cast<int *>(workspace);
  const int64_t items = (int64_t)E * ceil_div(N, GP::kM) * ceil_div(K, GP::kN);
  return dw_dtype == MOE_F32 ? launch_grouped<kWgradF32>(maps, g, items, stream)
                             : launch_grouped<kWgrad>(maps, g, items, stream);
}
