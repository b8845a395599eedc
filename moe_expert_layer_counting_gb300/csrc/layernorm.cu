// layernorm.cu -- layer norm with the residual stream's addition, and its
// gradients (include/moe_layernorm.h).
//
// Both directions are bound by HBM if the SM keeps up: every value is read once
// and written once, but a row needs its mean, then the squares of what is left
// after it (and two sums of gradients), and ~20 operations a value.
//   - A group of ceil(H / 512) warps owns a row at a time (two in the gradients),
//     a thread sixteen columns; groups walk the rows with a stride of all groups.  Of rows of up to 192 columns
//     a warp owns two or four (see lanes_of).
//   - A thread copies (cp.async) its own columns of the rows to come into its own
//     places in shared memory: the ring needs no barrier, only a wait for the
//     thread's own copies, and values are read from it again for each of a row's
//     steps, so that registers are left for the column sums.
//   - Arithmetic is on pairs (f32x2).
// The gradients' column sums are kept in registers over a block's rows, joined
// over its groups in shared memory, written as one part for each block and
// summed over the blocks, in a fixed order, by a second kernel.
// Measured (BF16, H = 7168): s and n of 8192 rows in 75 to 78 us (6.0 to 6.3 TB/s), of 4096 in 39;
// the gradients joined with ds of 8192 rows in 89 us (5.3 TB/s), of 4096 in 51, of which ~14 are the
// launch's start, its end, and the parts.  float32 rows: 123 us (5.7 TB/s) and 129 (6.4).
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "../../include/moe_layernorm.h"
#include "host_common.h"
#include "pairs.cuh"
#include "ptx.cuh"
#include "row_sums.cuh"

namespace mxq {

namespace {

constexpr int kMostH = 16384;

struct Rows {
  int64_t T;
  int H, warps, lanes, groups;            // warps of a group (a part of one: 1) and its threads, groups of a block
  int half;                               // gradients, kPair: columns of a cluster's first block
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

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's columns are runs of eight (BF16 rows) or four (float32 rows) of
// them, run r of thread t at column run * (r * threads of a group + t): 16 bytes a
// run of the rows' type, so that a warp's access is 512 bytes without gaps
// (with runs of eight float32 values: 157 instead of 132 us forward and 201 instead
// of 129 us for the gradients of 8192 x 7168).
template <typename XT> constexpr int kRun = 16 / sizeof(XT);
constexpr int kColumns = 16;              // of a thread

// BF16: a run of eight, or of four beside float32 rows.
template <int RUN>
__device__ __forceinline__ void copy_run(uint32_t dst, const uint16_t *src) {
  if (RUN == 8)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
template <int RUN>
__device__ __forceinline__ void copy_run(uint32_t dst, const float *src) {
  static_assert(RUN == 4, "16 bytes");
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int RUN>
__device__ __forceinline__ void take(const uint16_t *p, P2 (&v)[RUN / 2]) {
  if (RUN == 8) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    v[0] = from_bf16x2(a.x);
    v[1] = from_bf16x2(a.y);
    v[2 % (RUN / 2)] = from_bf16x2(a.z);
    v[3 % (RUN / 2)] = from_bf16x2(a.w);
  } else {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    v[0] = from_bf16x2(a.x);
    v[1] = from_bf16x2(a.y);
  }
}
template <int RUN>
__device__ __forceinline__ void take(const float *p, P2 (&v)[RUN / 2]) {
#pragma unroll
  for (int i = 0; i < RUN / 4; ++i) {
    const float4 a = reinterpret_cast<const float4 *>(p)[i];
    v[2 * i] = pair(a.x, a.y);
    v[2 * i + 1] = pair(a.z, a.w);
  }
}

template <int RUN>
__device__ __forceinline__ void put(uint16_t *p, const P2 (&v)[RUN / 2]) {
  if (RUN == 8)
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(to_bf16x2(v[0]), to_bf16x2(v[1]), to_bf16x2(v[2 % (RUN / 2)]), to_bf16x2(v[3 % (RUN / 2)]));
  else
    *reinterpret_cast<uint2 *>(p) = make_uint2(to_bf16x2(v[0]), to_bf16x2(v[1]));
}
template <int RUN>
__device__ __forceinline__ void put(float *p, const P2 (&v)[RUN / 2]) {
#pragma unroll
  for (int i = 0; i < RUN / 4; ++i) {
    const float2 a = split(v[2 * i]), b = split(v[2 * i + 1]);
    reinterpret_cast<float4 *>(p)[i] = make_float4(a.x, a.y, b.x, b.y);
  }
}

// A run of a weight of either type (the same branch for the whole launch).
template <int RUN>
__device__ __forceinline__ void weight(const void *w, int dtype, int col, P2 (&v)[RUN / 2]) {
  if (dtype == MOE_BF16)
    take<RUN>(static_cast<const uint16_t *>(w) + col, v);
  else
    take<RUN>(static_cast<const float *>(w) + col, v);
}

template <int N>
__device__ __forceinline__ P2 sum_of(const P2 (&v)[N]) {
  P2 s = v[0] + v[1];
#pragma unroll
  for (int i = 2; i < N; i += 2) s = s + (v[i] + v[i + 1]);
  return s;
}

__device__ __forceinline__ float both(P2 v) {
  const float2 f = split(v);
  return f.x + f.y;
}

// Sums over the `lanes` (8 or 16) threads that own a row, in each of them.
template <int N>
__device__ __forceinline__ void lanes_sum(float (&v)[N], int lanes) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
    if (o < lanes)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

// ---------------------------------------------------------------- forward

// Kinds of a launch: kShort rows of up to 192 columns, which a part of a warp owns; of more than 8192 columns kBig (forward) and
// kPair (gradients).
enum : int { kShort, kMiddle, kBig, kPair };

__device__ __forceinline__ void store_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// How the forward kernel goes about a launch: kRows rows of a group in work
// together, kSets sets of them in the ring (the next set's sum is added up with
// this one's squares: one exchange a set, and the sets after it are on their way).
// A row at a time and a deep ring, but for the shortest rows (BF16 without b), whose
// sums take longer than their bytes: 8192 x 7168 in 47 us by twos and 55 one by one;
// with b 84 by twos and 75 one by one.
//   BIG   rows of more than 8192 columns: 1024 threads of 64 registers, a row at a time, weights from L1.
template <typename XT, bool ADD, int KIND>
struct ForwardRing {
  static constexpr bool BIG = KIND == kBig;
  static constexpr int kSlot = kColumns * (int)(sizeof(XT) + (ADD ? 2 : 0));       // bytes of a thread's part of a row
  static constexpr int kThreads = BIG ? 1024 : 512;
  static constexpr int kRows = BIG || kSlot >= 64 ? 1 : 2;
  static constexpr int kSets = BIG ? (kSlot > 64 ? 2 : 3) : kSlot > 64 ? 4 : kSlot == 64 ? 6 : 3;
  static constexpr int kRed = 2 * 128 * 4;                   // bytes of a group's sums
  static size_t bytes(int threads, int tpr) {
    return (size_t)kSlot * kRows * kSets * threads + (tpr > 32 ? (size_t)(threads / tpr) * kRed : 0);
  }
};

template <typename XT, bool ADD, int KIND>
__global__ void __launch_bounds__(ForwardRing<XT, ADD, KIND>::kThreads, 1) layernorm_kernel(const Rows z) {
  using R = ForwardRing<XT, ADD, KIND>;
  constexpr bool BIG = KIND == kBig, SHORT = KIND == kShort;
  constexpr int RUN = kRun<XT>, kRuns = kColumns / RUN, kRows = R::kRows, kSets = R::kSets;
  extern __shared__ __align__(16) unsigned char ring[];      // [kSets][kRows] of [run][thread] of x, the same of b; sums
  const int threads = (int)blockDim.x, tpr = z.lanes;
  const int group = (int)threadIdx.x / tpr, t = (int)threadIdx.x - group * tpr;
  const int64_t stride = (int64_t)gridDim.x * z.groups;
  int64_t row = (int64_t)blockIdx.x * z.groups + group;
  const int sub = SHORT ? ((int)threadIdx.x & 31) / tpr : 0;           // of the warp's groups, whose rows follow one another
  float *red = reinterpret_cast<float *>(ring + kSets * kRows * R::kSlot * threads) + (SHORT ? 0 : group * (R::kRed / 4));
  if (z.warps > 1) {
    for (int i = t; i < R::kRed / 4; i += tpr) red[i] = 0.f;         // of warps that the group has not
    __syncthreads();
  }
  auto col = [&](int r) { return RUN * (r * tpr + t); };
  const uint32_t at = smem_u32(ring);
  // where run r of x and b lies in a slot
  auto of_x = [&](int slot, int r) { return slot * R::kSlot * threads + (r * threads + (int)threadIdx.x) * 16; };
  auto of_b = [&](int slot, int r) {
    return (slot * R::kSlot + kColumns * (int)sizeof(XT)) * threads + (r * threads + (int)threadIdx.x) * 2 * RUN;
  };
  pdl_launch_dependents();
  pdl_wait();
  auto send = [&](int64_t to_row, int set) {
#pragma unroll
    for (int j = 0; j < kRows; ++j, to_row += stride)
      if (to_row < z.T) {
#pragma unroll
        for (int r = 0; r < kRuns; ++r)
          if (col(r) < z.H) {
            copy_run<RUN>(at + of_x(set * kRows + j, r), static_cast<const XT *>(z.x) + to_row * z.ldx + col(r));
            if (ADD) copy_run<RUN>(at + of_b(set * kRows + j, r), z.b + to_row * z.ldb + col(r));
          }
      }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kSets; ++i) send(row + i * kRows * stride, i);
  P2 w[BIG ? 1 : kRuns][RUN / 2], bias[BIG ? 1 : kRuns][RUN / 2];
  if (!BIG) {
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
#pragma unroll
      for (int i = 0; i < RUN / 2; ++i) {
        w[BIG ? 0 : r][i] = twice(1.f);
        bias[BIG ? 0 : r][i] = twice(0.f);
      }
      if (z.w && col(r) < z.H) weight<RUN>(z.w, z.w_dtype, col(r), w[BIG ? 0 : r]);
      if (z.bias && col(r) < z.H) weight<RUN>(z.bias, z.w_dtype, col(r), bias[BIG ? 0 : r]);
    }
  }
  // run r of the row in a slot
  auto take_run = [&](int slot, int r, P2 (&v)[RUN / 2]) {
    take<RUN>(reinterpret_cast<const XT *>(ring + of_x(slot, r)), v);
    if (ADD) {
      P2 b[RUN / 2];
      take<RUN>(reinterpret_cast<const uint16_t *>(ring + of_b(slot, r)), b);
#pragma unroll
      for (int i = 0; i < RUN / 2; ++i) v[i] = v[i] + b[i];
    }
  };
  auto sum_row = [&](int slot) {
    P2 sum = twice(0.f);
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
      if (col(r) < z.H) {
        P2 v[RUN / 2];
        take_run(slot, r, v);
        sum = sum + sum_of(v);
      }
    return both(sum);
  };
  auto join = [&] {
    if (z.warps > 1)
      named_bar_sync(1 + group, 32 * z.warps);
    else
      __syncwarp();
  };
  copies_wait<kSets - 1>();
  float total[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) total[j] = row + j * stride < z.T ? sum_row(j) : 0.f;
  auto row_sum = [&](auto &v, float *where) {
    if (SHORT)
      lanes_sum(v, tpr);
    else
      group_sum(v, z.warps, t >> 5, where, join);
  };
  row_sum(total, red);
  int set = 0, turn = 0;
  for (; row - sub < z.T; row += kRows * stride) {
    const int after = set + 1 == kSets ? 0 : set + 1;
    P2 v[kRows][kRuns][RUN / 2];
    float sum[2 * kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const P2 mean = twice(-total[j] * z.inv_h);
      P2 sq = twice(0.f);
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
        if (col(r) < z.H) {
          P2(&u)[RUN / 2] = v[j][r];
          take_run(set * kRows + j, r, u);
          if (ADD && z.s && ((j == 0 && !SHORT) || row + j * stride < z.T))
            put<RUN>(static_cast<XT *>(z.s) + (row + j * stride) * z.lds + col(r), u);
#pragma unroll
          for (int i = 0; i < RUN / 2; ++i) {
            u[i] = u[i] + mean;
            sq = fma2(u[i], u[i], sq);
          }
        }
      sum[j] = both(sq);
    }
    copies_wait<kSets - 2>();
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      sum[kRows + j] = row + (kRows + j) * stride < z.T ? sum_row(after * kRows + j) : 0.f;
    turn ^= 1;                                               // a buffer is written again after the other's barrier
    row_sum(sum, red + turn * 128);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      total[j] = sum[kRows + j];
      if ((j > 0 || SHORT) && row + j * stride >= z.T) continue;
      const P2 rr = twice(rsqrtf(fmaf(sum[j], z.inv_h, z.eps)));
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
        if (col(r) < z.H) {
          P2(&u)[RUN / 2] = v[j][r];
          if (BIG) {
            P2 c[RUN / 2];
#pragma unroll
            for (int i = 0; i < RUN / 2; ++i) u[i] = u[i] * rr;
            if (z.w) {
              weight<RUN>(z.w, z.w_dtype, col(r), c);
#pragma unroll
              for (int i = 0; i < RUN / 2; ++i) u[i] = u[i] * c[i];
            }
            if (z.bias) {
              weight<RUN>(z.bias, z.w_dtype, col(r), c);
#pragma unroll
              for (int i = 0; i < RUN / 2; ++i) u[i] = u[i] + c[i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < RUN / 2; ++i) u[i] = fma2(u[i] * rr, w[BIG ? 0 : r][i], bias[BIG ? 0 : r][i]);
          }
          put<RUN>(z.n + (row + j * stride) * z.ldn + col(r), u);
        }
    }
    send(row + kSets * kRows * stride, set);
    set = after;
  }
}

// ---------------------------------------------------------------- gradients

// How the gradients' kernel goes about a launch.
//   kRows  rows of a group in work together: two, so that one's exchange and loads hide behind the other's
//          arithmetic (a block's 16 warps are all that fit: 32 column sums in registers); one where the ring
//          does not hold twice two.  4096 x 7168 in 51 us; 80 one by one, 75 with two blocks' worth of warps
//          at 72 registers.
//   kPair  rows of more than 8192 columns: a cluster of two blocks owns a row, half the columns each, and every
//          sum is joined through both blocks' shared memory, in one exchange a round, with the sums of the rows after
//          it (2048 x 16384, BF16 with ds, in 76 us; with two exchanges 83; one block of 1024 threads of 64 registers, a row at a time, 100).
template <typename XT, bool DS, int KIND>
struct GradRing {
  static constexpr int kSlot = kColumns * (int)(sizeof(XT) * (DS ? 2 : 1) + 2);    // bytes of a thread's part of a row
  static constexpr int kThreads = 512, kRows = kSlot > 96 ? 1 : 2;
  static constexpr int kRed = 2 * 8 * 32 * 4;                // bytes of a group's sums
  static size_t bytes(int threads, int tpr) {
    return (size_t)kSlot * 2 * kRows * threads + 4 * kColumns * tpr + (tpr > 32 ? (size_t)(threads / tpr) * kRed : 0);
  }
};

// Sums of N values over both blocks of a cluster, up to 16 warps each, the same bits in every thread; red [2 blocks][N][16] of
// each block, written again after another sum in another place.
template <int N>
__device__ __forceinline__ void pair_sum(float (&v)[N], uint32_t rank, float *red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (lane < 2) {
    const uint32_t to = mapa_shared(smem_u32(red + (int)rank * N * 16 + warp), (uint32_t)lane);
#pragma unroll
    for (int k = 0; k < N; ++k) store_cluster(to + 64 * k, v[k]);
  }
  cluster_sync();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = red[((lane >> 4) * N + k) * 16 + (lane & 15)];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

template <typename XT, bool DS, int KIND>
__global__ void __launch_bounds__(GradRing<XT, DS, KIND>::kThreads, 1) layernorm_grad_kernel(const Rows z) {
  using R = GradRing<XT, DS, KIND>;
  constexpr bool SHORT = KIND == kShort, PAIR = KIND == kPair;
  constexpr int RUN = kRun<XT>, kRuns = kColumns / RUN, kRows = R::kRows;
  // this block's columns: H from the first on
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int first = PAIR && rank ? z.half : 0, H = !PAIR ? z.H : rank ? z.H - z.half : z.half;
  const int64_t owner = PAIR ? blockIdx.x >> 1 : blockIdx.x, owners = PAIR ? gridDim.x >> 1 : gridDim.x;
  // [2][kRows] of [run][thread] of s, the same of dn and ds; w [run][thread of a group] in float32; the groups' sums.
  // At the end [2][H] floats.
  extern __shared__ __align__(16) unsigned char ring[];
  const int threads = (int)blockDim.x, tpr = z.lanes;
  const int group = (int)threadIdx.x / tpr, t = (int)threadIdx.x - group * tpr;
  const int64_t stride = owners * z.groups;
  int64_t row = owner * z.groups + group;
  float *const weights = reinterpret_cast<float *>(ring + 2 * kRows * R::kSlot * threads);
  const int sub = SHORT ? ((int)threadIdx.x & 31) / tpr : 0;           // of the warp's groups, whose rows follow one another
  float *red = weights + kColumns * tpr + (SHORT ? 0 : group * (R::kRed / 4));
  const uint32_t at = smem_u32(ring);
  auto col = [&](int r) { return RUN * (r * tpr + t); };
  auto of_s = [&](int slot, int r) { return slot * R::kSlot * threads + (r * threads + (int)threadIdx.x) * 16; };
  auto of_dn = [&](int slot, int r) {
    return (slot * R::kSlot + kColumns * (int)sizeof(XT)) * threads + (r * threads + (int)threadIdx.x) * 2 * RUN;
  };
  auto of_ds = [&](int slot, int r) {
    return (slot * R::kSlot + kColumns * (int)(sizeof(XT) + 2)) * threads + (r * threads + (int)threadIdx.x) * 16;
  };
  if (z.warps > 1)
    for (int i = t; i < R::kRed / 4; i += tpr) red[i] = 0.f;         // of warps that the group has not
  pdl_launch_dependents();
  pdl_wait();
  // rows to_row, to_row + stride, .. into half `half` of the ring
  auto send = [&](int64_t to_row, int half) {
#pragma unroll
    for (int j = 0; j < kRows; ++j, to_row += stride)
      if (to_row < z.T) {
#pragma unroll
        for (int r = 0; r < kRuns; ++r)
          if (col(r) < H) {
            const int slot = half * kRows + j;
            copy_run<RUN>(at + of_s(slot, r), static_cast<const XT *>(z.x) + to_row * z.ldx + first + col(r));
            copy_run<RUN>(at + of_dn(slot, r), z.b + to_row * z.ldb + first + col(r));
            if (DS) copy_run<RUN>(at + of_ds(slot, r), static_cast<const XT *>(z.ds) + to_row * z.ld_ds + first + col(r));
          }
      }
    copies_commit();
  };
  send(row, 0);
  send(row + kRows * stride, 1);
  // a group's weights in float32 (1 without w), the same for all groups
#pragma unroll
  for (int r = 0; r < kRuns; ++r)
    if (group == 0 && col(r) < H) {
      P2 w[RUN / 2];
#pragma unroll
      for (int i = 0; i < RUN / 2; ++i) w[i] = twice(1.f);
      if (z.w) weight<RUN>(z.w, z.w_dtype, first + col(r), w);
#pragma unroll
      for (int i = 0; i < RUN / 4; ++i) {
        const P2 two[2] = {w[2 * i], w[2 * i + 1]};
        put<4>(weights + ((r * RUN / 4 + i) * tpr + t) * 4, two);
      }
    }
  if (PAIR)
    cluster_sync();                    // and the other block's sums are zeroed
  else
    __syncthreads();
  auto take_w = [&](int r, P2 (&w)[RUN / 2]) {
#pragma unroll
    for (int i = 0; i < RUN / 4; ++i) {
      P2 two[2];
      take<4>(weights + ((r * RUN / 4 + i) * tpr + t) * 4, two);
      w[2 * i] = two[0];
      w[2 * i + 1] = two[1];
    }
  };
  auto join = [&] {
    if (z.warps > 1)
      named_bar_sync(1 + group, 32 * z.warps);
    else
      __syncwarp();
  };
  P2 dw[kRuns][RUN / 2], db[kRuns][RUN / 2];
#pragma unroll
  for (int r = 0; r < kRuns; ++r)
#pragma unroll
    for (int i = 0; i < RUN / 2; ++i) dw[r][i] = db[r][i] = twice(0.f);
  auto sum_rows = [&](int half, float *sum) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      P2 s = twice(0.f);
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
        if (col(r) < H) {
          P2 v[RUN / 2];
          take<RUN>(reinterpret_cast<const XT *>(ring + of_s(half * kRows + j, r)), v);
          s = s + sum_of(v);
        }
      sum[j] = both(s);
    }
  };
  float sum[kRows];
  if constexpr (PAIR) {
    copies_wait<1>();
    sum_rows(0, sum);
    pair_sum(sum, rank, red + 256);
  }
  // a row's sums go through two buffers, each written again after the other's barrier
  for (int half = 0; row - sub < z.T; half ^= 1) {
    const bool whole = kRows == 1 || row + stride < z.T;     // both rows are there
    const bool any = !SHORT || row < z.T;                    // the first is
    if constexpr (!PAIR) {
      copies_wait<1>();
      sum_rows(half, sum);
      if (SHORT)
        lanes_sum(sum, tpr);
      else
        group_sum(sum, z.warps, t >> 5, red, join);
    }
    P2 mean[kRows], sq[kRows], sg[kRows], sgv[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      mean[j] = twice(-sum[j] * z.inv_h);
      sq[j] = sg[j] = sgv[j] = twice(0.f);
    }
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
      if (col(r) < H) {
        P2 w[RUN / 2];
        take_w(r, w);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          P2 v[RUN / 2], d[RUN / 2];
          take<RUN>(reinterpret_cast<const XT *>(ring + of_s(half * kRows + j, r)), v);
          take<RUN>(reinterpret_cast<const uint16_t *>(ring + of_dn(half * kRows + j, r)), d);
#pragma unroll
          for (int i = 0; i < RUN / 2; ++i) {
            v[i] = v[i] + mean[j];
            const P2 g = d[i] * w[i];
            sq[j] = fma2(v[i], v[i], sq[j]);
            sg[j] = sg[j] + g;
            sgv[j] = fma2(g, v[i], sgv[j]);
          }
        }
      }
    float sums[kRows][3];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      sums[j][0] = both(sq[j]);
      sums[j][1] = both(sg[j]);
      sums[j][2] = both(sgv[j]);
    }
    if (SHORT) {
#pragma unroll
      for (int j = 0; j < kRows; ++j) lanes_sum(sums[j], tpr);
    } else if constexpr (PAIR) {
      // with the next rows' sums, so that a round has one exchange
      float all[4 * kRows];
#pragma unroll
      for (int k = 0; k < 3 * kRows; ++k) all[k] = sums[k / 3][k % 3];
      copies_wait<0>();
      sum_rows(half ^ 1, all + 3 * kRows);
      pair_sum(all, rank, red + 256 * half);
#pragma unroll
      for (int k = 0; k < 3 * kRows; ++k) sums[k / 3][k % 3] = all[k];
#pragma unroll
      for (int j = 0; j < kRows; ++j) sum[j] = all[3 * kRows + j];
    } else {
      group_sums(sums, z.warps, t >> 5, red + 256, join);
    }
    // dx = ds + r (g - mean(g)) - (v r) (r mean(g v) r): factor by factor, so that no power of a row's magnitude is formed
    P2 rr[kRows], mg[kRows], mgh[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const float q = rsqrtf(fmaf(sums[j][0], z.inv_h, z.eps));
      rr[j] = twice(q);
      mg[j] = twice(-sums[j][1] * z.inv_h);
      mgh[j] = twice(-(sums[j][2] * q) * z.inv_h);
    }
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
      if (col(r) < H) {
        P2 w[RUN / 2];
        take_w(r, w);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          if (j > 0 ? !whole : !any) break;
          P2 v[RUN / 2], d[RUN / 2], ds[RUN / 2], out[RUN / 2];
          take<RUN>(reinterpret_cast<const XT *>(ring + of_s(half * kRows + j, r)), v);
          take<RUN>(reinterpret_cast<const uint16_t *>(ring + of_dn(half * kRows + j, r)), d);
          if (DS) take<RUN>(reinterpret_cast<const XT *>(ring + of_ds(half * kRows + j, r)), ds);
#pragma unroll
          for (int i = 0; i < RUN / 2; ++i) {
            const P2 h = (v[i] + mean[j]) * rr[j];
            const P2 g = d[i] * w[i];
            dw[r][i] = fma2(d[i], h, dw[r][i]);
            db[r][i] = db[r][i] + d[i];
            const P2 a = fma2(h, mgh[j], g + mg[j]);
            out[i] = DS ? fma2(a, rr[j], ds[i]) : a * rr[j];
          }
          if (z.s) put<RUN>(static_cast<XT *>(z.s) + (row + j * stride) * z.lds + first + col(r), out);
        }
      }
    row += kRows * stride;
    send(row + kRows * stride, half);
  }
  if (!z.part) return;
  // a warp's groups' sums, then the groups' (warps') in their order
  if (SHORT)
    for (int o = tpr; o < 32; o <<= 1)
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
#pragma unroll
        for (int i = 0; i < RUN / 2; ++i) {
          const float2 a = split(dw[r][i]), b = split(db[r][i]);
          dw[r][i] = dw[r][i] + pair(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o));
          db[r][i] = db[r][i] + pair(__shfl_xor_sync(0xffffffffu, b.x, o), __shfl_xor_sync(0xffffffffu, b.y, o));
        }
  copies_wait<0>();
  __syncthreads();
  float *sums = reinterpret_cast<float *>(ring);
  const int part_of = SHORT ? (int)threadIdx.x >> 5 : group;
  for (int n = 0; n < (SHORT ? threads / 32 : z.groups); ++n) {
    if (part_of == n && sub == 0)
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
        if (col(r) < H)
#pragma unroll
          for (int i = 0; i < RUN / 2; ++i) {
            float2 *pw = reinterpret_cast<float2 *>(sums + col(r)) + i;
            float2 *pb = reinterpret_cast<float2 *>(sums + H + col(r)) + i;
            float2 a = split(dw[r][i]), b = split(db[r][i]);
            if (n > 0) {
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
  float *part = z.part + owner * 2 * z.H + first;
  for (int i = threadIdx.x; i < H / 2; i += threads) {
    const int of = i < H / 4 ? 0 : 1;                          // dw, dbias
    reinterpret_cast<float4 *>(part + (int64_t)of * z.H)[i - of * (H / 4)] = reinterpret_cast<const float4 *>(sums)[i];
  }
}

// Sums over the blocks' parts: 32 lanes a column each, kSumWarps warps share the parts, all loads of a thread in flight.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(32 * kSumWarps) sum_blocks_kernel(const float *part, int blocks, int H, float *dw, float *dbias) {
  __shared__ float red[kSumWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = (int)blockIdx.x * 32 + lane;                 // of 2 H
  float sum = 0.f;
  if (i < 2 * H)
#pragma unroll 8
    for (int b = warp; b < blocks; b += kSumWarps) sum += part[(int64_t)b * 2 * H + i];
  red[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || i >= 2 * H) return;
#pragma unroll
  for (int k = 1; k < kSumWarps; ++k) sum += red[k][lane];
  float *out = i < H ? dw : dbias;
  if (out) out[i < H ? i : i - H] = sum;
}

// ---------------------------------------------------------------- host

int warps_of(int64_t H) { return (int)ceil_div(H, 512); }
// Threads of a group.  Forward with b and gradients with ds, BF16, against a warp a row: 262 144 x 64 25 and 73 us (forward),
// 170 000 x 192 46 and 51, 59 and 65; 131 072 x 256 would be 48 and 46, 55 and 53.
int lanes_of(int64_t H) { return H <= 128 ? 8 : H <= 192 ? 16 : 32 * warps_of(H); }
constexpr int64_t kMostParts = 256;       // blocks of the gradients' kernel, one for each SM, at most

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

constexpr int kMostSmem = 227 * 1024;     // of a block

template <auto KERNEL>
int launch_rows(const Rows &z, int64_t blocks, size_t smem, cudaStream_t st, int cluster = 1) {
  static std::atomic<uint64_t> ready{0};                     // devices whose kernel attribute is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) != cudaSuccess) return MOE_ERR_CUDA;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)(z.lanes * z.groups));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, KERNEL, z) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
  z.lanes = lanes_of(a->H);
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
  auto launch_as = [&](auto type, auto with_b, auto kind) {
    using XT = decltype(type);
    using R = ForwardRing<XT, decltype(with_b)::value, decltype(kind)::value>;
    z.groups = std::max(1, R::kThreads / z.lanes);
    return launch_rows<layernorm_kernel<XT, decltype(with_b)::value, decltype(kind)::value>>(
        z, std::min<int64_t>(num_sms(), ceil_div(a->T, z.groups)), R::bytes(z.lanes * z.groups, z.lanes), stream);
  };
  auto launch = [&](auto type, auto with_b) {
    if (z.lanes < 32) return launch_as(type, with_b, std::integral_constant<int, kShort>{});
    return z.warps > 16 ? launch_as(type, with_b, std::integral_constant<int, kBig>{})
                        : launch_as(type, with_b, std::integral_constant<int, kMiddle>{});
  };
  using std::true_type;
  using std::false_type;
  if (a->x_dtype == MOE_F32) return a->b ? launch(0.f, true_type{}) : launch(0.f, false_type{});
  return a->b ? launch(uint16_t{0}, true_type{}) : launch(uint16_t{0}, false_type{});
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
  const bool pair = a->H > 8192;
  z.half = pair ? (int)round_up(ceil_div(a->H, 2), 8) : 0;
  z.warps = warps_of(pair ? z.half : a->H);
  z.lanes = lanes_of(pair ? z.half : a->H);
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
  int64_t parts = 0;
  auto launch_as = [&](auto type, auto with_ds, auto kind) {
    using XT = decltype(type);
    using R = GradRing<XT, decltype(with_ds)::value, decltype(kind)::value>;
    z.groups = std::max(1, R::kThreads / z.lanes);
    constexpr int cluster = decltype(kind)::value == kPair ? 2 : 1;
    parts = std::min({kMostParts, (int64_t)num_sms() / cluster, ceil_div(a->T, z.groups)});
    const size_t smem = std::max(R::bytes(z.lanes * z.groups, z.lanes), z.part ? (size_t)(pair ? z.half : z.H) * 8 : 0);
    return launch_rows<layernorm_grad_kernel<XT, decltype(with_ds)::value, decltype(kind)::value>>(z, cluster * parts, smem, stream, cluster);
  };
  const bool f32 = a->x_dtype == MOE_F32, add = a->ds != nullptr;
  auto launch = [&](auto type, auto with_ds) {
    if (pair) return launch_as(type, with_ds, std::integral_constant<int, kPair>{});
    return z.lanes < 32 ? launch_as(type, with_ds, std::integral_constant<int, kShort>{})
                        : launch_as(type, with_ds, std::integral_constant<int, kMiddle>{});
  };
  using std::true_type;
  using std::false_type;
  rc = f32 ? (add ? launch(0.f, true_type{}) : launch(0.f, false_type{}))
           : (add ? launch(uint16_t{0}, true_type{}) : launch(uint16_t{0}, false_type{}));
  if (rc != MOE_OK || !z.part) return rc;
  return launch_pdl(sum_blocks_kernel, dim3((unsigned)ceil_div(2 * z.H, 32)), dim3(32 * kSumWarps), 0, stream, z.part, (int)parts, z.H, a->dw,
                    a->dbias);
}
