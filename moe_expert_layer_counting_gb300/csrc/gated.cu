// gated.cu -- C entry points of the gated feed-forward block by expert
// (include/moe_gated.h): grouped_kernel.cuh's products with gated_epilogue.cuh's
// epilogues.
//
// forward.  A tile of the weights' rows holds 8 gate rows, then the 8 up rows of
// the same columns, and so on: one 5-D box per load brings them so, from the
// weights as they are.  Gate and up of a value then lie 8 TMEM lanes apart in
// one warp, and h costs a shuffle more than a plain product.  Against the product
// alone, h (and a, if asked for) is all that is written.
//
// dgrad.  The epilogue holds the gradient of h in float32, reads a once and
// writes da and h; dv is summed over 32 columns there and over the parts, in a
// fixed order, by a second small kernel.
#include "grouped_kernel.cuh"

namespace mxq {

namespace {

constexpr int kPartCols = 32;

// dv[r] = the sum of row r's parts, for the rows that an expert owns.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float *part, int parts, int64_t P, const int32_t *offsets,
                                                        int E, const int *status, float *dv) {
  pdl_launch_dependents();
  pdl_wait();
  if (status[0] != 0) return;                // bad offsets: no output
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (row < __ldg(offsets) || row >= __ldg(offsets + E)) return;
  float sum = 0.f;
#pragma unroll 8
  for (int i = 0; i < parts; ++i) sum += part[(int64_t)i * P + row];
  dv[row] = sum;
}

int check_gated(const moe_gated_args *a, bool back) {
  if (!a || a->struct_size != sizeof(moe_gated_args)) return MOE_ERR_INVALID_ARG;
  if (a->P < 0 || a->H <= 0 || a->I <= 0 || a->E <= 0) return MOE_ERR_INVALID_ARG;
  if (a->activation != MOE_ACT_SILU && a->activation != MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  if (a->P > 0x7fffffffLL || a->H > 0x7fffff00LL || a->I > 0x3fffff00LL || a->H % 8 != 0 || a->I % 8 != 0 ||
      a->E > kMaxExperts)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!a->offsets || !a->workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->workspace, 256) || !aligned(a->offsets, 4) || !aligned(a->row_w, 4) || !aligned(a->drow_w, 4))
    return MOE_ERR_MISALIGNED;
  if (a->workspace_bytes < moe_gated_workspace_size(a->P, a->H, a->I, a->E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!back && (a->da || a->drow_w)) return MOE_ERR_INVALID_ARG;
  if (a->P == 0) return MOE_OK;
  int rc = check_rows(a->rows, a->ld_rows, a->H);
  if (rc == MOE_OK && (back || a->a)) rc = check_rows(a->a, a->ld_a, 2 * a->I);
  if (rc == MOE_OK && (!back || a->h)) rc = check_rows(a->h, a->ld_h, a->I);
  if (rc == MOE_OK && back) rc = check_rows(a->da, a->ld_da, 2 * a->I);
  if (rc != MOE_OK) return rc;
  if (!a->w) return MOE_ERR_INVALID_ARG;
  return aligned(a->w, 16) ? MOE_OK : MOE_ERR_MISALIGNED;
}

// Gate and up rows of w [E][2I][H], 8 of each in turn, in boxes of 128.
bool encode_gated_weights(CUtensorMap *map, const uint16_t *w, uint64_t H, uint64_t I, uint64_t E) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[5] = {H, 8, 2, I / 8, E};
  const cuuint64_t strides[4] = {2 * H, 2 * H * I, 16 * H, 4 * H * I};
  const cuuint32_t box[5] = {(cuuint32_t)GP::kBK, 8, 2, 8, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<uint16_t *>(w), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int OP>
int gated_product(const moe_gated_args *a, cudaStream_t st) {
  constexpr bool kBack = OP == kGatedGrad;
  const int rc = check_gated(a, kBack);
  if (rc != MOE_OK) return rc;
  if (a->P == 0) return cudaMemsetAsync(a->workspace, 0, 64, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  GMaps maps;
  bool ok = kBack ? encode_map(&maps.a, a->w, 3, a->I, a->H, a->E, a->I, a->H * a->I, 64, GP::kBK)
                  : encode_gated_weights(&maps.a, a->w, a->H, a->I, a->E);
  for (int i = 0; i < 5; ++i)
    ok = ok && encode_map(&maps.b[i], a->rows, 2, a->H, a->P, 1, a->ld_rows, 0, GP::kBK, kBoxRows[i]);
  if (!ok) return MOE_ERR_CUDA;
  GArgs g{};
  g.offsets = a->offsets;
  g.P = a->P;
  g.E = a->E;
  g.M = (int)(kBack ? a->I : 2 * a->I);
  g.R = (int)a->H;
  g.inject_wait = injected_wait();
  g.status = reinterpret_cast<int *>(a->workspace);
  float *part = kBack && a->drow_w ? reinterpret_cast<float *>(static_cast<char *>(a->workspace) + kStatusBytes) : nullptr;
  g.gated = {(int)a->I, a->activation, a->row_w, a->a, a->ld_a, a->h, a->ld_h, a->da, a->ld_da, part};
  const int64_t tiles = std::min<int64_t>(a->P, a->P / GP::kN + a->E);
  const int launched = launch_grouped<OP>(maps, g, tiles * ceil_div(g.M, GP::kM), st);
  if (launched != MOE_OK || !part) return launched;
  return launch_pdl(sum_parts_kernel, dim3((unsigned)ceil_div(a->P, 256)), dim3(256), 0, st, part,
                    (int)ceil_div(a->I, kPartCols), a->P, a->offsets, (int)a->E, g.status, a->drow_w);
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" size_t moe_gated_workspace_size(int64_t P, int64_t H, int64_t I, int32_t E) {
  if (P < 0 || H <= 0 || I <= 0 || E <= 0) return 0;
  return kStatusBytes + round_up((size_t)P * (size_t)ceil_div(I, kPartCols) * 4, 256);
}

extern "C" int moe_gated_forward(const moe_gated_args *args, cudaStream_t stream) {
  return gated_product<kGated>(args, stream);
}

extern "C" int moe_gated_dgrad(const moe_gated_args *args, cudaStream_t stream) {
  return gated_product<kGatedGrad>(args, stream);
}
