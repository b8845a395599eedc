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

// ---------------------------------------------------------------- few rows

// forward of up to kFewRows rows: products of matrices and a few vectors, bound by the weights' way from HBM.
// A warp takes one gate row and its up row whole, all their loads in flight at
// once, and the rows of x that belong to the expert from L1: every SM has work, where
// the tensor cores' tiles of 256 weight rows are fewer than SMs, and no pair of SMs
// is waited for.  Which calls: see few_rows_win().
constexpr int kFewRows = 8, kFewWarps = 8;

__device__ __forceinline__ uint4 load_once(const uint16_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b, float sum) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), sum);
    sum = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), sum);
  }
  return sum;
}

struct FewArgs {
  const uint16_t *x, *w;
  int64_t ldx, H;
  const int32_t *offsets;
  int P, E;
  int *status;
  GatedArgs gated;
};

// Column i of rows row0 .. row0 + rows - 1 (at most ROWS) of expert e.
template <int ROWS>
__device__ __forceinline__ void few_rows(const FewArgs &g, int e, int row0, int rows, int i, int lane) {
  constexpr int kUnroll = ROWS == 1 ? 8 : ROWS == 2 ? 4 : 2;
  const uint16_t *gate = g.w + ((int64_t)e * 2 * g.gated.I + i) * g.H, *up = gate + (int64_t)g.gated.I * g.H;
  const uint16_t *x[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) x[r] = g.x + (int64_t)(row0 + min(r, rows - 1)) * g.ldx;
  float a[ROWS], b[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) a[r] = b[r] = 0.f;
  for (int64_t k0 = 8 * lane; k0 < g.H; k0 += 256 * kUnroll) {
    uint4 wg[kUnroll], wu[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      wg[j] = wu[j] = make_uint4(0, 0, 0, 0);
      if (k0 + 256 * j < g.H) {
        wg[j] = load_once(gate + k0 + 256 * j);
        wu[j] = load_once(up + k0 + 256 * j);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (k0 + 256 * j < g.H)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const uint4 v = __ldg(reinterpret_cast<const uint4 *>(x[r] + k0 + 256 * j));
          a[r] = dot8(wg[j], v, a[r]);
          b[r] = dot8(wu[j], v, b[r]);
        }
  }
  float ga = 0.f, gb = 0.f;            // lane r: row r's
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a[r] += __shfl_xor_sync(0xffffffffu, a[r], o);
      b[r] += __shfl_xor_sync(0xffffffffu, b[r], o);
    }
    if (lane == r) {
      ga = a[r];
      gb = b[r];
    }
  }
  if (lane >= rows) return;            // (of an inlined call: on to the warp's next column)
  const int64_t row = row0 + lane;
  const float v = g.gated.row_w ? __ldg(g.gated.row_w + row) : 1.f;
  float dq;
  const float h = ga * gate_sigmoid(g.gated.activation, ga, dq) * gb * v;
  reinterpret_cast<__nv_bfloat16 *>(g.gated.h)[row * g.gated.ld_h + i] = __float2bfloat16_rn(h);
  if (g.gated.a) {
    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(g.gated.a) + row * g.gated.ld_a + i;
    out[0] = __float2bfloat16_rn(ga);
    out[g.gated.I] = __float2bfloat16_rn(gb);
  }
}

__global__ void __launch_bounds__(32 * kFewWarps, 2) gated_few_kernel(const FewArgs g) {
  __shared__ int expert[kFewRows], runs;
  __shared__ int4 run[kFewRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < kFewRows) expert[threadIdx.x] = -1;
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  const bool first = blockIdx.x == 0;
  if (first && threadIdx.x < 16) g.status[threadIdx.x] = 0;
  int bad = 0;
  for (int e = threadIdx.x; e <= g.E; e += 32 * kFewWarps) {
    const int o = __ldg(g.offsets + e), before = e > 0 ? __ldg(g.offsets + e - 1) : 0;
    if (o < before || o > g.P) {
      bad = 1;
    } else if (e > 0) {
      for (int r = max(before, 0); r < o; ++r) expert[r] = e - 1;      // before <= r < o <= P <= kFewRows
    }
  }
  if (__syncthreads_or(bad)) {
    if (first && threadIdx.x == 0) report_status(g.status, kStatusBadIndex);
    return;
  }
  // experts with rows, each a run of rows
  if (threadIdx.x == 0) {
    int n = 0;
    for (int r = 0; r < g.P; ++r) {
      const int e = expert[r];
      if (e < 0) continue;
      if (n > 0 && run[n - 1].x == e) {
        ++run[n - 1].z;
      } else {
        run[n++] = make_int4(e, r, 1, 0);
      }
    }
    runs = n;
  }
  __syncthreads();
  const int total = runs * g.gated.I;
  for (int u = (int)blockIdx.x * kFewWarps + warp; u < total; u += (int)gridDim.x * kFewWarps) {
    const int n = u / g.gated.I, i = u - n * g.gated.I;
    const int e = run[n].x, row0 = run[n].y, rows = run[n].z;
    if (rows == 1)
      few_rows<1>(g, e, row0, rows, i, lane);
    else if (rows == 2)
      few_rows<2>(g, e, row0, rows, i, lane);
    else if (rows <= 4)
      few_rows<4>(g, e, row0, rows, i, lane);
    else
      few_rows<8>(g, e, row0, rows, i, lane);
  }
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

// Few rows, here against the tensor cores' kernel (I x H, us, graph replay): one dense block 512 x 2048, one row 4.3 and
// 8.8, eight rows 8.2 and 8.8; 2048 x 7168, one row 14.4 and 18.2, two 15.2, four 17.9, eight 25 and 18.2 (arithmetic); 8
// rows of 8 of 256 experts, 512 x 2048, 10.7 and 12.1, 2048 x 7168 (470 MB of weights) 89 and 73 (fewer bytes in flight).
bool few_rows_win(const moe_gated_args *a) {
  const int64_t most = std::min<int64_t>(a->P, a->E);           // experts with rows
  return a->P <= kFewRows && (a->E > 1 || a->P <= 2) && most * 4 * a->I * a->H <= (96LL << 20);
}

template <int OP>
int gated_product(const moe_gated_args *a, cudaStream_t st) {
  constexpr bool kBack = OP == kGatedGrad;
  const int rc = check_gated(a, kBack);
  if (rc != MOE_OK) return rc;
  if (a->P == 0) return cudaMemsetAsync(a->workspace, 0, 64, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  if (!kBack && few_rows_win(a)) {
    const FewArgs few{a->rows, a->w, a->ld_rows, a->H, a->offsets, (int)a->P, (int)a->E, reinterpret_cast<int *>(a->workspace),
                      {(int)a->I, a->activation, a->row_w, a->a, a->ld_a, a->h, a->ld_h, nullptr, 0, nullptr}};
    const int64_t units = std::min<int64_t>(a->P, a->E) * a->I;
    return launch_pdl(gated_few_kernel, dim3((unsigned)std::min<int64_t>(2 * num_sms(), ceil_div(units, kFewWarps))),
                      dim3(32 * kFewWarps), 0, st, few);
  }
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
