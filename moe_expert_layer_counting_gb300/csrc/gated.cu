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
// A block takes eight columns of h, so eight gate and the eight up rows, its warps a share of the sums each. Every SM has
// work, where the tiles of 256 weight rows are fewer than SMs, and no pair of SMs is waited for.
// A warp's mma (m16n8k16: the one whose operands are registers, as the weights go through once) has the gate rows as rows
// 0 to 7, the up rows as 8 to 15 and the rows of x as columns, so that a lane ends with gate and up of the same
// values. The sum's order is free, so that a lane's 16 bytes of a row are two mma's operands as they are loaded.
// Which calls: see few_rows_win().
constexpr int kFewRows = 16, kFewWarps = 8;

__device__ __forceinline__ uint4 load_once(const uint16_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t gate0, uint32_t up0, uint32_t gate1, uint32_t up1, uint32_t x0,
                                         uint32_t x1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(gate0), "r"(up0), "r"(gate1), "r"(up1), "r"(x0), "r"(x1));
}

struct FewArgs {
  const uint16_t *x, *w;
  int64_t ldx, H;
  const int32_t *offsets;
  int P, E;
  int *status;
  GatedArgs gated;
};

// Columns i0 .. i0 + 7 of rows row0 .. row0 + rows - 1 (at most 8 TILES) of expert e, by a block; red [warps][4 TILES][32].
template <int TILES>
__device__ __forceinline__ void few_rows(const FewArgs &g, int e, int row0, int rows, int i0, float *red) {
  constexpr int kUnroll = TILES == 1 ? 6 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int of = lane >> 2;                            // the lane's weight row, and its row of x in each tile
  const int64_t first = 32 * warp + 8 * (lane & 3);
  const uint16_t *gate = g.w + ((int64_t)e * 2 * g.gated.I + i0 + of) * g.H, *up = gate + (int64_t)g.gated.I * g.H;
  const uint16_t *x[TILES];
  float d[TILES][4];
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    x[t] = g.x + (int64_t)(row0 + min(8 * t + of, rows - 1)) * g.ldx;
    d[t][0] = d[t][1] = d[t][2] = d[t][3] = 0.f;
  }
  for (int64_t base = 0; base < g.H; base += 32 * kFewWarps * kUnroll) {
    uint4 wg[kUnroll], wu[kUnroll], v[kUnroll][TILES];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int64_t k = base + first + 32 * kFewWarps * j;
      wg[j] = wu[j] = make_uint4(0, 0, 0, 0);
      if (k < g.H) {
        wg[j] = load_once(gate + k);
        wu[j] = load_once(up + k);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int64_t k = base + first + 32 * kFewWarps * j;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        v[j][t] = make_uint4(0, 0, 0, 0);
        if (k < g.H) v[j][t] = __ldg(reinterpret_cast<const uint4 *>(x[t] + k));
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        mma_16x8(d[t], wg[j].x, wu[j].x, wg[j].y, wu[j].y, v[j][t].x, v[j][t].y);
        mma_16x8(d[t], wg[j].z, wu[j].z, wg[j].w, wu[j].w, v[j][t].z, v[j][t].w);
      }
  }
  // of a tile: d[0], d[1] gate row `of` with rows 2 (lane % 4) and the next of x; d[2], d[3] the up row
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int c = 0; c < 4; ++c) red[(warp * 4 * TILES + 4 * t + c) * 32 + lane] = d[t][c];
  __syncthreads();
  if (warp >= 2 * TILES) return;             // warp: of a tile's gates, the first or the second (of an inlined call: on)
  const int t = warp >> 1, c = warp & 1;
  const int r = 8 * t + 2 * (lane & 3) + c, i = i0 + of;
  if (r >= rows) return;
  float ga = 0.f, gb = 0.f;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) {
    ga += red[(w * 4 * TILES + 4 * t + c) * 32 + lane];
    gb += red[(w * 4 * TILES + 4 * t + 2 + c) * 32 + lane];
  }
  const int64_t row = row0 + r;
  const float scale = g.gated.row_w ? __ldg(g.gated.row_w + row) : 1.f;
  float dq;
  const float h = ga * gate_sigmoid(g.gated.activation, ga, dq) * gb * scale;
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
  __shared__ float red[2][kFewWarps * 4 * (kFewRows / 8) * 32];        // a unit writes one while the last's is read
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
  const int across = g.gated.I / 8, total = runs * across;
  int turn = 0;
  for (int u = (int)blockIdx.x; u < total; u += (int)gridDim.x, turn ^= 1) {
    const int n = u / across, i0 = 8 * (u - n * across);
    const int e = run[n].x, row0 = run[n].y, rows = run[n].z;
    if (rows <= 8)
      few_rows<1>(g, e, row0, rows, i0, red[turn]);
    else
      few_rows<2>(g, e, row0, rows, i0, red[turn]);
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

// Few rows, here against the tensor cores' tiles (I x H, us, graph replay): one dense block 512 x 2048, one row 4.4 and 8.8,
// eight 5.2 and 8.8, sixteen 6.1 and 8.8; 2048 x 7168 11.5, 12.4, 13.9 and 18.2; 4096 x 8192 (134 MB of weights) 23, 24,
// 26.3 and 25.6. 8 rows of 8 of 256 experts, 512 x 2048, 9.9 and 11.9, of 64, 2048 x 7168 (470 MB), 70.4 and 70.8;
// 16 of 16, 512 x 2048 (67 MB), 17.0 and 16.5. So up to eight rows always, more while their weights are few.
bool few_rows_win(const moe_gated_args *a) {
  const int64_t most = std::min<int64_t>(a->P, a->E);           // experts with rows
  return a->P <= 8 || (a->P <= kFewRows && most * 4 * a->I * a->H <= (64LL << 20));
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
    const int64_t units = std::min<int64_t>(a->P, a->E) * (a->I / 8);
    return launch_pdl(gated_few_kernel, dim3((unsigned)std::min<int64_t>(2 * num_sms(), units)),
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
  const int64_t items = most_row_items(g);
  const int launched = part && a->H > kDvBlocks * GP::kBK ? launch_grouped<kBack ? kGatedGradDv : OP>(maps, g, items, st)
                                                          : launch_grouped<OP>(maps, g, items, st);
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
