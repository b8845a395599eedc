// layernorm.cu -- layer norm with the residual stream's addition, and its
// gradients (include/moe_layernorm.h).
//
// Both directions are bound by HBM: every value is read once and written once.
// A group of ceil(H / 512) warps owns a row at a time, a thread two runs of
// eight columns; groups walk the rows with a stride of all groups.  A thread
// copies (cp.async) its own columns of the rows to come into its own places in
// shared memory, so that the ring needs no barrier: it waits for its own copies,
// takes them into registers, and sends the places' next copies on their way
// before the row's first sum.  The mean comes first and the squares of what is
// left after it second, both from registers: two sums a row over the group, in
// the gradients one and three.  Arithmetic is on pairs (f32x2).
//
// The gradients' column sums are kept in registers over a block's rows, joined
// over its groups in shared memory, written as one part for each block and
// summed over the blocks, in a fixed order, by a second kernel.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "../../include/moe_layernorm.h"
#include "host_common.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace mxq {

namespace {

constexpr int kMostH = 16384;
constexpr int kBlock = 512;               // threads of a block where a row's group is no larger

struct Rows {
  int64_t T;
  int H, warps, groups;                   // warps of a group, groups of a block
  int w_dtype;
  float eps, inv_h;
  const void *x, *w, *bias;
  const uint16_t *b;                      // forward: b; gradients: dn
  const void *ds;
  int64_t ldx, ldb, ld_ds;
  void *s;                                // forward: s; gradients: dx
  uint16_t *n;
  int64_t lds, ldn;
  float *part;                            // gradients: [blocks][2][H], or NULL
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16-byte pieces of a run of eight values.
template <typename T> constexpr int kPieces = sizeof(T) == 2 ? 1 : 2;

template <typename T>
__device__ __forceinline__ void take8(const uint4 *place, int threads, P2 (&v)[4]) {
  const uint4 a = place[0];
  if (sizeof(T) == 2) {
    v[0] = from_bf16x2(a.x);
    v[1] = from_bf16x2(a.y);
    v[2] = from_bf16x2(a.z);
    v[3] = from_bf16x2(a.w);
  } else {
    const uint4 b = place[threads];
    v[0] = pair(__uint_as_float(a.x), __uint_as_float(a.y));
    v[1] = pair(__uint_as_float(a.z), __uint_as_float(a.w));
    v[2] = pair(__uint_as_float(b.x), __uint_as_float(b.y));
    v[3] = pair(__uint_as_float(b.z), __uint_as_float(b.w));
  }
}

template <typename T>
__device__ __forceinline__ void put8(T *p, const P2 (&v)[4]) {
  if (sizeof(T) == 2) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(to_bf16x2(v[0]), to_bf16x2(v[1]), to_bf16x2(v[2]), to_bf16x2(v[3]));
  } else {
    const float2 a = split(v[0]), b = split(v[1]), c = split(v[2]), d = split(v[3]);
    reinterpret_cast<float4 *>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
  }
}

// Eight values of a weight of either type.
__device__ __forceinline__ void weight8(const void *w, int dtype, int col, P2 (&v)[4]) {
  if (dtype == MOE_BF16) {
    const uint4 q = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + col));
    v[0] = from_bf16x2(q.x);
    v[1] = from_bf16x2(q.y);
    v[2] = from_bf16x2(q.z);
    v[3] = from_bf16x2(q.w);
  } else {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + col);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = pair(a.x, a.y);
    v[1] = pair(a.z, a.w);
    v[2] = pair(b.x, b.y);
    v[3] = pair(b.z, b.w);
  }
}

// Sums over the group, the same bits in every thread.  `red`: of this group and
// of this place in a row (a place's words are written again only after the row's
// other sum, whose barrier every reader has passed by then).
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int warps, int group, float (*red)[N]) {
  const int lane = (int)(threadIdx.x & 31);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (warps == 1) return;
  const int warp = (int)(threadIdx.x >> 5) - group * warps;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) red[warp][k] = v[k];
  named_bar_sync(1 + group, 32 * warps);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = lane < warps ? red[lane][k] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

__device__ __forceinline__ float both(P2 v) {
  const float2 f = split(v);
  return f.x + f.y;
}

// ---------------------------------------------------------------- forward

template <typename XT, bool ADD>
__global__ void __launch_bounds__(1024, 1) layernorm_kernel(const Rows z) {
  constexpr int kP = kPieces<XT>, kPer = 2 * kP + (ADD ? 2 : 0), kDepth = 2;
  extern __shared__ __align__(16) uint4 ring[];              // [depth][piece][thread]
  __shared__ float red[2][32][1];
  const int threads = (int)blockDim.x, tpr = 32 * z.warps;
  const int group = (int)threadIdx.x / tpr, t = (int)threadIdx.x - group * tpr;
  const int col[2] = {8 * t, 8 * (tpr + t)};
  const bool has[2] = {col[0] < z.H, col[1] < z.H};
  uint4 *mine = ring + threadIdx.x;
  const uint32_t at = smem_u32(mine);
  const int64_t first = (int64_t)blockIdx.x * z.groups + group, stride = (int64_t)gridDim.x * z.groups;
  pdl_launch_dependents();
  pdl_wait();
  auto send = [&](int64_t row, int slot) {
    if (row < z.T) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (has[c]) {
          const XT *x = static_cast<const XT *>(z.x) + row * z.ldx + col[c];
          const uint32_t to = at + (uint32_t)(slot * kPer * threads) * 16;
#pragma unroll
          for (int p = 0; p < kP; ++p) copy16(to + (uint32_t)((c * kP + p) * threads) * 16, reinterpret_cast<const uint4 *>(x) + p);
          if (ADD) copy16(to + (uint32_t)((2 * kP + c) * threads) * 16, z.b + row * z.ldb + col[c]);
        }
    }
    copies_commit();
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) send(first + d * stride, d);
  int slot = 0;
  for (int64_t row = first; row < z.T; row += stride) {
    copies_wait<kDepth - 1>();
    P2 v[2][4];
    const uint4 *place = mine + slot * kPer * threads;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (has[c]) {
        take8<XT>(place + c * kP * threads, threads, v[c]);
        if (ADD) {
          P2 b[4];
          take8<uint16_t>(place + (2 * kP + c) * threads, threads, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][i] = v[c][i] + b[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = twice(0.f);
      }
    }
    send(row + kDepth * stride, slot);
    slot ^= 1;
    if (ADD && z.s) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (has[c]) put8<XT>(static_cast<XT *>(z.s) + row * z.lds + col[c], v[c]);
    }
    float sum[1] = {both(((v[0][0] + v[0][1]) + (v[0][2] + v[0][3])) + ((v[1][0] + v[1][1]) + (v[1][2] + v[1][3])))};
    group_sums<1>(sum, z.warps, group, red[0] + (z.warps > 1 ? group * z.warps : 0));
    const P2 mean = twice(-sum[0] * z.inv_h);
    P2 sq = twice(0.f);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[c][i] = v[c][i] + mean;
        if (has[c]) sq = fma2(v[c][i], v[c][i], sq);
      }
    sum[0] = both(sq);
    group_sums<1>(sum, z.warps, group, red[1] + (z.warps > 1 ? group * z.warps : 0));
    const P2 r = twice(rsqrtf(fmaf(sum[0], z.inv_h, z.eps)));
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (has[c]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = v[c][i] * r;
        P2 w[4];
        if (z.w) {
          weight8(z.w, z.w_dtype, col[c], w);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][i] = v[c][i] * w[i];
        }
        if (z.bias) {
          weight8(z.bias, z.w_dtype, col[c], w);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][i] = v[c][i] + w[i];
        }
        put8<uint16_t>(z.n + row * z.ldn + col[c], v[c]);
      }
  }
}

// ---------------------------------------------------------------- gradients

// BIG: rows of more than 8192 columns, 64 registers a thread.
template <typename XT, bool DS, bool BIG>
__global__ void __launch_bounds__(BIG ? 1024 : kBlock, 1) layernorm_grad_kernel(const Rows z) {
  constexpr int kP = kPieces<XT>, kPer = 2 * kP + 2 + (DS ? 2 * kP : 0), kDepth = BIG && sizeof(XT) == 4 ? 1 : 2;
  extern __shared__ __align__(16) uint4 ring[];              // [depth][piece][thread]; at the end [2][H] floats
  __shared__ float red1[32][1], red3[32][3];
  const int threads = (int)blockDim.x, tpr = 32 * z.warps;
  const int group = (int)threadIdx.x / tpr, t = (int)threadIdx.x - group * tpr;
  const int col[2] = {8 * t, 8 * (tpr + t)};
  const bool has[2] = {col[0] < z.H, col[1] < z.H};
  uint4 *mine = ring + threadIdx.x;
  const uint32_t at = smem_u32(mine);
  const int64_t first = (int64_t)blockIdx.x * z.groups + group, stride = (int64_t)gridDim.x * z.groups;
  const int of_group = z.warps > 1 ? group * z.warps : 0;
  pdl_launch_dependents();
  pdl_wait();
  auto send = [&](int64_t row, int slot) {
    if (row < z.T) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (has[c]) {
          const uint32_t to = at + (uint32_t)(slot * kPer * threads) * 16;
          const XT *x = static_cast<const XT *>(z.x) + row * z.ldx + col[c];
#pragma unroll
          for (int p = 0; p < kP; ++p) copy16(to + (uint32_t)((c * kP + p) * threads) * 16, reinterpret_cast<const uint4 *>(x) + p);
          copy16(to + (uint32_t)((2 * kP + c) * threads) * 16, z.b + row * z.ldb + col[c]);
          if (DS) {
            const XT *ds = static_cast<const XT *>(z.ds) + row * z.ld_ds + col[c];
#pragma unroll
            for (int p = 0; p < kP; ++p)
              copy16(to + (uint32_t)((2 * kP + 2 + c * kP + p) * threads) * 16, reinterpret_cast<const uint4 *>(ds) + p);
          }
        }
    }
    copies_commit();
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) send(first + d * stride, d);
  P2 dw[2][4], db[2][4];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[c][i] = db[c][i] = twice(0.f);
  int slot = 0;
  for (int64_t row = first; row < z.T; row += stride) {
    copies_wait<kDepth - 1>();
    P2 v[2][4], d[2][4], ds[DS ? 2 : 1][4];
    const uint4 *place = mine + slot * kPer * threads;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (has[c]) {
        take8<XT>(place + c * kP * threads, threads, v[c]);
        take8<uint16_t>(place + (2 * kP + c) * threads, threads, d[c]);
        if (DS) take8<XT>(place + (2 * kP + 2 + c * kP) * threads, threads, ds[DS ? c : 0]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = d[c][i] = ds[DS ? c : 0][i] = twice(0.f);
      }
    }
    send(row + kDepth * stride, slot);
    if (kDepth == 2) slot ^= 1;
    float sum[1] = {both(((v[0][0] + v[0][1]) + (v[0][2] + v[0][3])) + ((v[1][0] + v[1][1]) + (v[1][2] + v[1][3])))};
    group_sums<1>(sum, z.warps, group, red1 + of_group);
    const P2 mean = twice(-sum[0] * z.inv_h);
    P2 sq = twice(0.f), sg = twice(0.f), sgv = twice(0.f);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (has[c]) {
        P2 w[4];
        if (z.w) weight8(z.w, z.w_dtype, col[c], w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[c][i] = v[c][i] + mean;
          const P2 g = z.w ? d[c][i] * w[i] : d[c][i];
          sq = fma2(v[c][i], v[c][i], sq);
          sg = sg + g;
          sgv = fma2(g, v[c][i], sgv);
        }
      }
    float sums[3] = {both(sq), both(sg), both(sgv)};
    group_sums<3>(sums, z.warps, group, red3 + of_group);
    const float r = rsqrtf(fmaf(sums[0], z.inv_h, z.eps));
    // dx = ds + r (g - mean(g)) - (v r) (r mean(g v) r): factor by factor, so that no power of a row's magnitude is formed
    const P2 rr = twice(r), mg = twice(-sums[1] * z.inv_h), mgh = twice(-(sums[2] * r) * z.inv_h);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (has[c]) {
        P2 w[4], out[4];
        if (z.w) weight8(z.w, z.w_dtype, col[c], w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const P2 h = v[c][i] * rr;
          const P2 g = z.w ? d[c][i] * w[i] : d[c][i];
          dw[c][i] = fma2(d[c][i], h, dw[c][i]);
          db[c][i] = db[c][i] + d[c][i];
          const P2 a = fma2(h, mgh, g + mg);
          out[i] = DS ? fma2(a, rr, ds[DS ? c : 0][i]) : a * rr;
        }
        if (z.s) put8<XT>(static_cast<XT *>(z.s) + row * z.lds + col[c], out);
      }
  }
  if (!z.part) return;
  // the groups' sums, joined in their order
  copies_wait<0>();
  __syncthreads();
  float *sums = reinterpret_cast<float *>(ring);
  for (int k = 0; k < z.groups; ++k) {
    if (group == k)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (has[c])
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 *pw = reinterpret_cast<float2 *>(sums + col[c]) + i, *pb = reinterpret_cast<float2 *>(sums + z.H + col[c]) + i;
            float2 a = split(dw[c][i]), b = split(db[c][i]);
            if (k > 0) {
              a.x += pw->x;
              a.y += pw->y;
              b.x += pb->x;
              b.y += pb->y;
            }
            *pw = a;
            *pb = b;
          }
    __syncthreads();
  }
  float4 *part = reinterpret_cast<float4 *>(z.part + (int64_t)blockIdx.x * 2 * z.H);
  for (int i = threadIdx.x; i < z.H / 2; i += threads) part[i] = reinterpret_cast<const float4 *>(sums)[i];
}

// Sums over the blocks' parts: 32 lanes a column each, 8 warps share the parts.
__global__ void __launch_bounds__(256) sum_blocks_kernel(const float *part, int blocks, int H, float *dw, float *dbias) {
  __shared__ float red[8][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = (int)blockIdx.x * 32 + lane;                 // of 2 H
  float sum = 0.f;
  if (i < 2 * H)
#pragma unroll 8
    for (int b = warp; b < blocks; b += 8) sum += part[(int64_t)b * 2 * H + i];
  red[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || i >= 2 * H) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) sum += red[k][lane];
  float *out = i < H ? dw : dbias;
  if (out) out[i < H ? i : i - H] = sum;
}

// ---------------------------------------------------------------- host

int warps_of(int64_t H) { return (int)ceil_div(H, 512); }
int groups_of(int64_t H) { return std::max(1, kBlock / (32 * warps_of(H))); }
// Blocks of the gradients' kernel: one for each SM, its rows' column sums in its registers.
constexpr int64_t kMostParts = 256;
int64_t grad_blocks(int64_t T, int64_t H) { return std::min({kMostParts, (int64_t)num_sms(), ceil_div(T, groups_of(H))}); }

int check_rows_of(const void *p, int64_t ld, int64_t H) {
  if (!p || ld < H) return MOE_ERR_INVALID_ARG;
  if (ld % 8 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  return aligned(p, 16) ? MOE_OK : MOE_ERR_MISALIGNED;
}

int check_sizes(int64_t T, int64_t H, int32_t x_dtype, int32_t w_dtype, float eps) {
  if (T < 0 || H <= 0 || (x_dtype != MOE_BF16 && x_dtype != MOE_F32) || (w_dtype != MOE_BF16 && w_dtype != MOE_F32) ||
      !(eps >= 0.f) || std::isinf(eps))
    return MOE_ERR_INVALID_ARG;
  return H % 8 != 0 || H > kMostH || T > 0x7fffffffffLL ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

template <auto KERNEL>
int launch_rows(const Rows &z, int64_t blocks, int pieces_deep, size_t least_smem, cudaStream_t st) {
  constexpr int kMostSmem = 230 * 1024 - 4096;               // beside the kernels' static words
  static std::atomic<uint64_t> ready{0};                     // devices whose kernel attribute is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) != cudaSuccess) return MOE_ERR_CUDA;
    ready.fetch_or(bit, std::memory_order_release);
  }
  const int threads = 32 * z.warps * z.groups;
  const size_t smem = std::max((size_t)pieces_deep * threads * 16, least_smem);
  return launch_pdl(KERNEL, dim3((unsigned)blocks), dim3((unsigned)threads), smem, st, z);
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" size_t moe_layernorm_workspace_size(int64_t T, int64_t H) {
  if (T < 0 || H <= 0 || H > kMostH) return 0;
  return round_up((size_t)std::max<int64_t>(1, std::min(T, kMostParts)) * 2 * (size_t)H * 4, 256);
}

extern "C" int moe_layernorm_forward(const moe_layernorm_args *a, cudaStream_t stream) {
  if (!a || a->struct_size != sizeof(moe_layernorm_args)) return MOE_ERR_INVALID_ARG;
  int rc = check_sizes(a->T, a->H, a->x_dtype, a->w_dtype, a->eps);
  if (rc != MOE_OK) return rc;
  if (!a->b && a->s) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->w, 16) || !aligned(a->bias, 16)) return MOE_ERR_MISALIGNED;
  if (a->T == 0) return MOE_OK;
  if ((rc = check_rows_of(a->x, a->ldx, a->H)) != MOE_OK || (a->b && (rc = check_rows_of(a->b, a->ldb, a->H)) != MOE_OK) ||
      (a->s && (rc = check_rows_of(a->s, a->lds, a->H)) != MOE_OK) || (rc = check_rows_of(a->n, a->ldn, a->H)) != MOE_OK)
    return rc;
  Rows z{};
  z.T = a->T;
  z.H = (int)a->H;
  z.warps = warps_of(a->H);
  z.groups = groups_of(a->H);
  z.w_dtype = a->w_dtype;
  z.eps = a->eps;
  z.inv_h = 1.f / (float)a->H;
  z.x = a->x;
  z.ldx = a->ldx;
  z.b = a->b;
  z.ldb = a->ldb;
  z.w = a->w;
  z.bias = a->bias;
  z.s = a->s;
  z.lds = a->lds;
  z.n = a->n;
  z.ldn = a->ldn;
  const int64_t per_sm = z.warps * z.groups > 16 ? 1 : 2;
  const int64_t blocks = std::min<int64_t>(per_sm * num_sms(), ceil_div(a->T, z.groups));
  const int deep = 2 * (2 * (a->x_dtype == MOE_BF16 ? 1 : 2) + (a->b ? 2 : 0));
  if (a->x_dtype == MOE_BF16)
    return a->b ? launch_rows<layernorm_kernel<uint16_t, true>>(z, blocks, deep, 0, stream)
                : launch_rows<layernorm_kernel<uint16_t, false>>(z, blocks, deep, 0, stream);
  return a->b ? launch_rows<layernorm_kernel<float, true>>(z, blocks, deep, 0, stream)
              : launch_rows<layernorm_kernel<float, false>>(z, blocks, deep, 0, stream);
}

extern "C" int moe_layernorm_backward(const moe_layernorm_grads *a, cudaStream_t stream) {
  if (!a || a->struct_size != sizeof(moe_layernorm_grads)) return MOE_ERR_INVALID_ARG;
  int rc = check_sizes(a->T, a->H, a->x_dtype, a->w_dtype, a->eps);
  if (rc != MOE_OK) return rc;
  if (a->dw && !a->w) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->w, 16) || !aligned(a->dw, 16) || !aligned(a->dbias, 16) || !aligned(a->workspace, 256))
    return MOE_ERR_MISALIGNED;
  if (a->dw || a->dbias) {
    if (!a->workspace) return MOE_ERR_INVALID_ARG;
    if (a->workspace_bytes < moe_layernorm_workspace_size(a->T, a->H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  if (a->T == 0) {
    for (float *sum : {a->dw, a->dbias})
      if (sum && cudaMemsetAsync(sum, 0, (size_t)a->H * 4, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if ((rc = check_rows_of(a->s, a->lds, a->H)) != MOE_OK || (rc = check_rows_of(a->dn, a->ld_dn, a->H)) != MOE_OK ||
      (a->ds && (rc = check_rows_of(a->ds, a->ld_ds, a->H)) != MOE_OK) ||
      (a->dx && (rc = check_rows_of(a->dx, a->ld_dx, a->H)) != MOE_OK))
    return rc;
  if (!a->dx && !a->dw && !a->dbias) return MOE_OK;
  Rows z{};
  z.T = a->T;
  z.H = (int)a->H;
  z.warps = warps_of(a->H);
  z.groups = groups_of(a->H);
  z.w_dtype = a->w_dtype;
  z.eps = a->eps;
  z.inv_h = 1.f / (float)a->H;
  z.x = a->s;
  z.ldx = a->lds;
  z.b = a->dn;
  z.ldb = a->ld_dn;
  z.w = a->w;
  z.ds = a->ds;
  z.ld_ds = a->ld_ds;
  z.s = a->dx;
  z.lds = a->ld_dx;
  z.part = a->dw || a->dbias ? static_cast<float *>(a->workspace) : nullptr;
  const int64_t blocks = grad_blocks(a->T, a->H);
  const bool big = z.warps > 16, f32 = a->x_dtype == MOE_F32, add = a->ds != nullptr;
  const int pieces = 2 * (f32 ? 2 : 1) * (add ? 2 : 1) + 2, deep = pieces * (big && f32 ? 1 : 2);
  const size_t least = z.part ? (size_t)z.H * 8 : 0;
  auto launch = [&](auto type, auto with_ds) {
    using XT = decltype(type);
    constexpr bool kDs = decltype(with_ds)::value;
    return big ? launch_rows<layernorm_grad_kernel<XT, kDs, true>>(z, blocks, deep, least, stream)
               : launch_rows<layernorm_grad_kernel<XT, kDs, false>>(z, blocks, deep, least, stream);
  };
  using std::true_type;
  using std::false_type;
  rc = f32 ? (add ? launch(0.f, true_type{}) : launch(0.f, false_type{}))
           : (add ? launch(uint16_t{0}, true_type{}) : launch(uint16_t{0}, false_type{}));
  if (rc != MOE_OK || !z.part) return rc;
  return launch_pdl(sum_blocks_kernel, dim3((unsigned)ceil_div(2 * z.H, 32)), dim3(256), 0, stream, z.part, (int)blocks, z.H, a->dw,
                    a->dbias);
}
