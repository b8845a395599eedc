// muon.cu -- matrices orthogonalised by Newton-Schulz products, and a step of
// Muon over a stack of them (include/moe_muon.h).
//
// An iteration X = (a + b G + c G^2) X with G = X X^T is three products over the
// shorter side n.  Completing the square,
//   a + b G + c G^2 = c S^2 + (a - b^2 / 4c),   S = G + b / 2c,
// makes each of them a plain product with a factor and a number on the diagonal:
//   S = X X^T + b/2c      (symmetric: tiles on and above the diagonal, each
//   Q = c S S + a - b^2/4c  stored twice)
//   X = Q X
// so that no epilogue reads a second matrix, and the values that are rounded, S,
// are small where X is nearly orthogonal.  In all n^2 k + n^3 + 2 n^2 k operations
// instead of 4 n^2 k + 2 n^3.
//
// FP16 iterates.  All singular values of an iterate are below 1.3, so that its
// range is known and FP16 with a fixed scale of 2^12 (16 at most, 2^-26 the
// smallest normal value) keeps 11 bits where BF16 keeps 8, at the same rate.
// The diagonals of S and Q alone are kept in full (left_of): rounded, they would
// be off by nearly the same in every row, which is as much as all else together
// (1024 x 2048: 1.6e-3 of the result instead of 7e-4, 30 x 3383 3.2e-3 instead of
// 6e-4; the times are the same).
//
// Measured: 64 matrices of 1024 x 2048, five iterations: 1.87 to 2.07 ms in a burst (two
// GPUs; 1.29 to 1.16 PFLOP/s of 7.5 GFLOP a matrix and iteration; the tiles on the
// diagonal add a tenth to that), 2.25 back to back at the power limit (1.5 GHz); a step of 8 of 7168 x 2048 with
// float32 masters and copies 2.7 to 3.2 ms, of which 0.5 are the three passes over the values at 7 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdlib>

#include "../../include/moe_muon.h"
#include "grouped_kernel.cuh"

namespace mxq {

namespace {

constexpr float kScale = 4096.f;           // of every FP16 matrix
constexpr int kMostParts = 1024;           // partial sums of a matrix's squares

// ---------------------------------------------------------------- momentum, norm, scaling

struct Elementwise {
  int64_t E, N, K, ld;      // ld: row stride of the FP16 matrices
  int parts, per;           // blocks of a matrix, values of a block (a multiple of 8)
  const void *g;            // gradient, or the matrices themselves
  int g_dtype;
  float *m;                 // NULL: orthogonalise g
  const float *grad_scale;
  float mu, gain;           // gain: 1 - mu
  int nesterov;
  float eps;
  float *sums;              // [E][parts]
  uint16_t *x;              // [E][N][ld]
  int *status;
  int *sync;                // [1 + E] of the products, zeroed by the first kernel
  // the end
  void *p;
  int p_dtype;
  uint16_t *copy;
  int update;               // 1: p = keep p - rate X; 0: p = X
  float keep, rate;
};

template <int VEC>
__device__ __forceinline__ void load_values(const void *p, int dtype, int64_t i, float (&v)[VEC]) {
  if (VEC == 8) {
    if (dtype == MOE_BF16) {
      const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    } else {
      const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
      const float4 a = q[0], b = q[1];
      const float t[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[k] = t[k];
    }
  } else {
    v[0] = dtype == MOE_BF16 ? bf16_bits_to_float(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
  }
}

template <int VEC>
__device__ __forceinline__ void store_values(void *p, int dtype, int64_t i, const float (&v)[VEC]) {
  if (VEC == 8) {
    if (dtype == MOE_BF16) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
      q[0] = make_float4(v[0], v[1 % VEC], v[2 % VEC], v[3 % VEC]);
      q[1] = make_float4(v[4 % VEC], v[5 % VEC], v[6 % VEC], v[7 % VEC]);
    }
  } else if (dtype == MOE_BF16) {
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v[0]);
  } else {
    static_cast<float *>(p)[i] = v[0];
  }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Where X has value i of matrix e.
__device__ __forceinline__ int64_t place_of(const Elementwise &z, int64_t e, int64_t i) {
  if (z.ld == z.K) return e * z.N * z.K + i;
  const int64_t r = i >> 32 ? i / z.K : (int64_t)((uint32_t)i / (uint32_t)z.K);
  return (e * z.N + r) * z.ld + (i - r * z.K);
}

// The sum over the block, in every thread (256 threads; a fixed order).
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += red[i];
  return v;
}

// What is orthogonalised, at value i: the gradient or, after the momentum's update, u.
// `fresh`: m is still the momentum before this step.
template <int VEC>
__device__ __forceinline__ void values_of(const Elementwise &z, int64_t i, float gs, bool fresh, float (&u)[VEC]) {
  load_values<VEC>(z.g, z.g_dtype, i, u);
  if (!z.m) return;
  float m[VEC];
  load_values<VEC>(z.m, MOE_F32, i, m);
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const float g = z.gain * (u[k] * gs);
    if (fresh) m[k] = fmaf(z.mu, m[k], g);
    u[k] = z.nesterov ? fmaf(z.mu, m[k], g) : m[k];
  }
  if (fresh) store_values<VEC>(z.m, MOE_F32, i, m);
}

// m's update and the squares' sum of each part of each matrix.
template <int VEC>
__global__ void __launch_bounds__(256) momentum_kernel(const Elementwise z) {
  __shared__ float red[8];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t e = blockIdx.y, size = z.N * z.K;
  if (blockIdx.x == 0 && e == 0 && threadIdx.x < 16) z.status[threadIdx.x] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    z.sync[1 + e] = 0;
    if (e == 0) z.sync[0] = 0;
  }
  const float gs = z.grad_scale ? *z.grad_scale : 1.f;
  const int64_t i0 = (int64_t)blockIdx.x * z.per, i1 = min(i0 + z.per, size);
  float sum = 0.f;
#pragma unroll 2
  for (int64_t i = i0 + threadIdx.x * VEC; i < i1; i += 256 * VEC) {
    float u[VEC];
    values_of<VEC>(z, e * size + i, gs, true, u);
#pragma unroll
    for (int k = 0; k < VEC; ++k) sum = fmaf(u[k], u[k], sum);
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) z.sums[e * z.parts + blockIdx.x] = sum;
}

// X = u / max(|u|, eps) in FP16.
template <int VEC>
__global__ void __launch_bounds__(256) scale_kernel(const Elementwise z) {
  __shared__ float red[8];
  pdl_launch_dependents();
  pdl_wait();
  // backwards: what the kernel before touched last is still in L2
  const int64_t e = gridDim.y - 1 - blockIdx.y, size = z.N * z.K;
  const int part = (int)(gridDim.x - 1 - blockIdx.x);
  float sum = 0.f;
  for (int i = threadIdx.x; i < z.parts; i += 256) sum += z.sums[e * z.parts + i];
  sum = block_sum(sum, red);
  // (max written so that a NaN stays one)
  const float norm = sqrtf(sum), by = norm == 0.f ? 0.f : kScale / (norm < z.eps ? z.eps : norm);
  const float gs = z.grad_scale ? *z.grad_scale : 1.f;
  const int64_t i0 = (int64_t)part * z.per, i1 = min(i0 + z.per, size);
#pragma unroll 2
  for (int64_t i = i0 + threadIdx.x * VEC; i < i1; i += 256 * VEC) {
    float u[VEC];
    values_of<VEC>(z, e * size + i, gs, false, u);
    if (VEC == 8) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) w[k] = pack_f16(u[2 * k] * by, u[2 * k + 1] * by);
      *reinterpret_cast<uint4 *>(z.x + place_of(z, e, i)) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      reinterpret_cast<__half *>(z.x)[place_of(z, e, i)] = __float2half_rn(u[0] * by);
    }
  }
}

// p = keep p - rate X, and its copy.
template <int VEC>
__global__ void __launch_bounds__(256) update_kernel(const Elementwise z) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t e = blockIdx.y, size = z.N * z.K;
  const int64_t i0 = (int64_t)blockIdx.x * z.per, i1 = min(i0 + z.per, size);
  const float rate = (z.update ? z.rate : -1.f) * (1.f / kScale);
#pragma unroll 2
  for (int64_t i = i0 + threadIdx.x * VEC; i < i1; i += 256 * VEC) {
    float x[VEC], p[VEC];
    if (VEC == 8) {
      const uint4 q = *reinterpret_cast<const uint4 *>(z.x + place_of(z, e, i));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    } else {
      x[0] = __half2float(reinterpret_cast<const __half *>(z.x)[place_of(z, e, i)]);
    }
    if (z.update) {
      load_values<VEC>(z.p, z.p_dtype, e * size + i, p);
#pragma unroll
      for (int k = 0; k < VEC; ++k) p[k] = fmaf(-rate, x[k], z.keep * p[k]);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) p[k] = -rate * x[k];
    }
    store_values<VEC>(z.p, z.p_dtype, e * size + i, p);
    if (z.copy) store_values<VEC>(z.copy, MOE_BF16, e * size + i, p);
  }
}

// ---------------------------------------------------------------- products

// All products of a call in one launch.  Products of one kind over the stack are a
// stage: S = alpha A B^T + beta on the diagonal, and so on; a tile of a stage of
// one matrix is an item.  Pairs of CTAs (M = 256, N up to 256 per item; 64
// reduction values a stage of the ring, two accumulators) claim items in
// order, iteration by iteration, stage by stage.  An item may begin when the
// stages before it are done with its matrix: each of its tiles has raised
// the matrix's counter then.  Items are claimed in order and depend on earlier ones only, so
// that the earliest one in work never waits, whatever part of the grid is
// resident.  Against a launch for each product: 8 matrices of 256 x 128 in 62 us instead
// of 85, a step of 8 of 1000 x 520 in 160 instead of 224; large ones the same.
struct NsStage {
  int M, C, R;              // rows and columns of the result, length of the sums
  int a_mn, b_mn;           // the operand's M (N) index is the contiguous one in memory (else the summed one)
  int symmetric;            // the result is: tiles on and above the diagonal, each stored twice
  int tn, items;            // columns of a tile; tiles of a matrix
  float alpha, beta;
  uint16_t *d;              // symmetric: the result
  int64_t ld;
};

// 10 maps of [E][rows][columns]: boxes of 128 rows and of 32 rows x 64 columns, and of 64 x 64.
struct NsMaps {
  CUtensorMap x128[2], x32[2], x64[2], s128, s32, q128, q32;
};

struct NsArgs {
  NsStage stage[3];         // Gram matrix to S (without c: to Q), Q from S, X from Q and X
  int E, steps, wide, square;       // wide: N <= K; square: the second stage is there
  int *ticket, *done;       // next item; [E] warps that are done with a tile
  float *of_s, *of_q;       // [E][ld_of]: what FP16 leaves of the diagonals (see left_of)
  int ld_of;                // a multiple of 64
  int inject_wait;
  int *status;
};

struct NsLayout {
  static constexpr int kStages = 6, kSlot = 32768, kEpiBytes = 4096;
  static constexpr int kClaims = 2, kAhead = 8;     // items in the ring; blocks before an item's last that the next is claimed
  static constexpr int kOffEpi = kStages * kSlot;
  static constexpr int kOffItems = kOffEpi + GP::kEpiWarps * kEpiBytes;
  static constexpr int kOffOf = kOffItems + 16 * kClaims;          // 256 floats: what is left of a diagonal, for a tile's drain
  static constexpr int kOffBar = kOffOf + 4 * GP::kN;
  static constexpr int kNumBars = 2 * kStages + 7 + 2 * kClaims + 2;
  static constexpr int kOffTmemPtr = (kOffBar + 8 * kNumBars + 63) & ~63;
  static constexpr int kBytes = 1024 + kOffTmemPtr + 64;
};
static_assert(NsLayout::kBytes <= 232448, "shared memory of one CTA");

struct NsItem {
  int e, m, c, at;          // at: 3 * iteration + stage; -1 after the last
  bool ready;               // the matrix is known to be ready
};
constexpr int kNsReady = 1 << 16;          // in the ring: beside at

// Packed words turned as turn_bf16 turns floats: word i of a lane holds rows 2 i and
// 2 i + 1 of its column.
template <int NW, typename Put>
__device__ __forceinline__ void turn_words(const uint32_t *v, int lane, Put put) {
  const bool b0 = (lane & 1) != 0, b1 = (lane & 2) != 0, b2 = (lane & 4) != 0;
  uint32_t w[NW];                      // rows 2 i + b0, two columns
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, v[i], 1);
    w[i] = __byte_perm(v[i], got, b0 ? 0x3276 : 0x5410);
  }
  uint32_t u[NW / 2][2];               // rows 4 q + 2 b1 + b0, four columns
#pragma unroll
  for (int q = 0; q < NW / 2; ++q) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? w[2 * q] : w[2 * q + 1], 2);
    u[q][0] = b1 ? got : w[2 * q];
    u[q][1] = b1 ? w[2 * q + 1] : got;
  }
#pragma unroll
  for (int r = 0; r < NW / 4; ++r) {
    const uint32_t got0 = __shfl_xor_sync(0xffffffffu, b2 ? u[2 * r][0] : u[2 * r + 1][0], 4);
    const uint32_t got1 = __shfl_xor_sync(0xffffffffu, b2 ? u[2 * r][1] : u[2 * r + 1][1], 4);
    put(r, b2 ? make_uint4(got0, got1, u[2 * r + 1][0], u[2 * r + 1][1])
              : make_uint4(u[2 * r][0], u[2 * r][1], got0, got1));
  }
}

__device__ __forceinline__ uint32_t make_idesc_f16(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
  return make_idesc_bf16(m, n, a_mn, b_mn) & ~((7u << 7) | (7u << 10));      // A and B: FP16 is 0
}

// Items of a ring that one thread fills and every role of both CTAs reads.
struct NsItems {
  const int4 *items;
  uint64_t *full;
  uint32_t empty0;          // the leader's barriers, shared::cluster
  int *status;
  int slot;
  uint32_t phase;

  // `wide`: called by a warp, not by a thread
  __device__ __forceinline__ bool next(NsItem &it, bool wide) {
    const bool got = mbar_wait_reset(full + slot, phase, status, kLimit, kWaitArrival, slot);
    if (!(wide ? __all_sync(0xffffffffu, got) : got)) return false;
    const int4 v = items[slot];
    it = NsItem{v.x, v.y, v.z, v.w < 0 ? -1 : v.w & (kNsReady - 1), (v.w & kNsReady) != 0};
    if (wide) __syncwarp();
    if (!wide || (threadIdx.x & 31) == 0) mbar_arrive_done(empty0 + 8 * (uint32_t)slot);
    if (++slot == NsLayout::kClaims) { slot = 0; phase ^= 1; }
    return it.at >= 0;
  }
};

__device__ __forceinline__ void store_cluster_v4(uint32_t addr, int4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Item w of the launch.
__device__ __forceinline__ int4 ns_item(const NsArgs &g, int64_t w) {
  const int per[3] = {g.stage[0].items, g.square ? g.stage[1].items : 0, g.stage[2].items};
  const int64_t iteration = (int64_t)g.E * (per[0] + per[1] + per[2]);
  const int it = (int)(w / iteration);
  if (it >= g.steps) return make_int4(0, 0, 0, -1);
  int64_t r = w - it * iteration;
  int k = 0;
  while (k < 2 && r >= (int64_t)g.E * per[k]) {
    r -= (int64_t)g.E * per[k];
    ++k;
  }
  const NsStage &s = g.stage[k];
  const int e = (int)(r / per[k]);
  int i = (int)(r - (int64_t)e * per[k]), m = 0;
  const int ct = (s.C + s.tn - 1) / s.tn;
  if (s.symmetric) {
    // row m of tiles begins at the diagonal
    const int across = GP::kM / s.tn;
    while (i >= ct - m * across) {
      i -= ct - m * across;
      ++m;
    }
    i += m * across;
  } else {
    m = i / ct;
    i -= m * ct;
  }
  return make_int4(e, m, i, 3 * it + k);
}

// As wait_counter, with a quick look before it: the stages of small matrices are a
// few microseconds apart.
__device__ __forceinline__ bool ns_wait(const int *counter, int target, int *status, int pos) {
  for (int i = 0; i < 64; ++i)
    if (ld_acquire_gpu(counter) >= target) return true;
  return wait_counter(counter, target, status, kLimit, pos);
}

// Arrivals at a matrix's counter before stage `at` of it may begin.
__device__ __forceinline__ int ns_arrivals(const NsArgs &g, int at) {
  const int it = at / 3, k = at - 3 * it;
  const int a = g.stage[0].items, b = g.square ? g.stage[1].items : 0, c = g.stage[2].items;
  return 2 * GP::kEpiWarps * (it * (a + b + c) + (k > 0 ? a : 0) + (k > 1 ? b : 0));
}

// What FP16 leaves of a diagonal's value x (both scaled).  Of S: what it adds to Q's diagonal, 2 c h (x - h).  Of Q: the factor of
// X's row (of tall matrices, column) that stands for it, as the other values of a row add up to little beside it.  A stage's
// drain writes them, the next one's reads them: the thread of the loads fetches them behind its last load (fetched by the drain's
// warps, after the accumulator: chains of short stages 5 to 8 % slower; with a wait of these warps for the matrix: 12 %).
__device__ __forceinline__ float left_of(float x, bool of_square, float square_alpha) {
  const float h = __half2float(__float2half_rn(x));
  return of_square ? 2.f * square_alpha * h * (x - h) : h == 0.f ? 1.f : __fdividef(x, h);
}

// Whether a tile's drain needs values of of_s (its rows', for Q's diagonal) or of of_q (X's rows', of tall matrices columns').
__device__ __forceinline__ bool needs_of(const NsItem &it, const NsStage &s, int k) {
  return k == 2 || (k == 1 && it.c * s.tn < (it.m + 1) * GP::kM);
}

__device__ __forceinline__ int tile_slots(const NsStage &s, int c) { return min(s.tn, (s.C - c * s.tn + 31) & ~31); }

__global__ void __launch_bounds__(GP::kThreads, 1) newton_schulz_kernel(const __grid_constant__ NsMaps maps,
                                                                        const __grid_constant__ NsArgs g) {
  using L = NsLayout;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);      // leader: both CTAs' copies of a stage
  uint64_t *empty = full + L::kStages;                                   // each CTA: stage consumed
  uint64_t *tmem_full = empty + L::kStages;                              // each CTA: accumulator ready
  uint64_t *tmem_empty = tmem_full + 2;                                  // leader: both CTAs drained it
  uint64_t *mma_done = tmem_empty + 2;
  uint64_t *never = mma_done + 1;
  uint64_t *item_full = never + 1;                                       // each CTA
  uint64_t *item_empty = item_full + L::kClaims;                         // leader: both CTAs' roles have read it
  uint64_t *want = item_empty + L::kClaims;                              // leader: its loads are nearly done
  uint64_t *of_full = want + 1, *of_empty = of_full + 1;                 // each CTA: values for a drain, read by its warps
  int4 *ring = reinterpret_cast<int4 *>(smem + L::kOffItems);
  uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(smem + L::kOffTmemPtr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  int *status = g.status;

  if (warp == 0) {
    if (lane < 10) tma_prefetch_desc(&maps.x128[0] + lane);
  } else if (warp == 2) {
    if (lane == 0) {
      for (int s = 0; s < L::kStages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      for (int a = 0; a < 2; ++a) {
        mbar_init(&tmem_full[a], 1);
        mbar_init(&tmem_empty[a], 2 * GP::kEpiWarps);
      }
      mbar_init(mma_done, 1);
      mbar_init(never, 1);
      mbar_init(want, 1);
      mbar_init(of_full, 1);
      mbar_init(of_empty, GP::kEpiWarps);
      for (int c = 0; c < L::kClaims; ++c) {
        mbar_init(item_full + c, 1);
        mbar_init(item_empty + c, 2 + 2 * GP::kEpiWarps + 1);      // loads, epilogues, the leader's MMAs
      }
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc_2sm(tmem_ptr, 512);
    tmem_relinquish_2sm();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t tmem_base = *tmem_ptr;
  NsItems items{ring, item_full, mapa_shared(smem_u32(item_empty), 0), status, 0, 0};
  NsItem it;

  if (warp == 0) {
    // ------------------------------------------------------------ loads (both CTAs), one thread
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0, ofs = 0;           // ofs: drains' values fetched so far
      bool ok = true;
      const uint32_t full0 = mapa_shared(smem_u32(full), 0);
      const uint64_t policy = l2_policy(false);
      while (ok && items.next(it, false)) {
        const int iteration = it.at / 3, k = it.at - 3 * iteration, x = iteration & 1;
        const NsStage &s = g.stage[k];
        const int n = tile_slots(s, it.c), half = n >> 1, blocks = (s.R + GP::kBK - 1) / GP::kBK;
        const int row = it.m * GP::kM + (int)rank * 128, col = it.c * s.tn + (int)rank * half;
        // a: Gram matrix X, square S, product Q or (tall) X; b: X, S, X or (tall) Q
        const bool is_x_a = k == 0 || (k == 2 && !g.wide), is_x_b = k == 0 || (k == 2 && g.wide);
        const CUtensorMap *a_map = is_x_a ? (s.a_mn ? &maps.x64[x] : &maps.x128[x]) : k == 1 ? &maps.s128 : &maps.q128;
        const CUtensorMap *b_map = is_x_b ? (s.b_mn ? &maps.x64[x] : half > 64 ? &maps.x128[x] : &maps.x32[x])
                                   : k == 1 ? (half > 64 ? &maps.s128 : &maps.s32)
                                            : (half > 64 ? &maps.q128 : &maps.q32);
        // rows of a box of b, and boxes
        const int b_box = s.b_mn ? 64 : half > 64 ? 128 : 32, b_boxes = (half + b_box - 1) / b_box;
        const uint32_t bytes = (uint32_t)(GP::kATile + b_boxes * b_box * GP::kBK * 2);
        if (!it.ready) ok = ns_wait(g.done + it.e, ns_arrivals(g, it.at), status, it.at);
        fence_proxy_async_global();       // what was stored from registers is read by TMA
        for (int kb = 0; kb < blocks && ok; ++kb) {
          unsigned char *a = smem + stage * L::kSlot, *b = a + GP::kATile;
          const uint32_t bar = full0 + 8 * (uint32_t)stage;
          const int k0 = kb * GP::kBK;
          ok = mbar_wait_reset(&empty[stage], phase ^ 1, status, kLimit, kWaitProducerEmpty, kb);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
          if (s.a_mn) {
#pragma unroll
            for (int j = 0; j < 2; ++j) tma_load_3d_2sm(a + j * GP::kHalfBox, a_map, bar, row + 64 * j, k0, it.e, policy);
          } else {
            tma_load_3d_2sm(a, a_map, bar, k0, row, it.e, policy);
          }
          for (int j = 0; j < b_boxes; ++j) {
            if (s.b_mn)
              tma_load_3d_2sm(b + j * GP::kHalfBox, b_map, bar, col + 64 * j, k0, it.e, policy);
            else
              tma_load_3d_2sm(b + j * b_box * GP::kBK * 2, b_map, bar, k0, col + b_box * j, it.e, policy);
          }
          if (rank == 0 && kb == max(0, blocks - L::kAhead)) mbar_arrive(want);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == L::kStages) { stage = 0; phase ^= 1; }
        }
        if (ok && needs_of(it, s, k)) {
          // after the tile's loads: the drain before this one may still read its own
          const bool columns = k == 2 && !g.wide;
          const uint32_t of_bytes = 4u * (columns ? s.tn : 128);                  // (past a row's end: the next one's)
          ok = mbar_wait_reset(of_empty, (ofs & 1) ^ 1, status, kLimit, kWaitProducerEmpty, it.at);
          if (ok) {
            mbar_arrive_expect_tx(of_full, of_bytes);
            bulk_load(smem + L::kOffOf, (k == 1 ? g.of_s : g.of_q) + (int64_t)it.e * g.ld_of + (columns ? it.c * s.tn : row), of_bytes,
                      of_full);
            ++ofs;
          }
        }
      }
      // no CTA leaves with copies in flight (as in grouped_kernel)
      for (int s = 0; s < L::kStages; ++s)
        if (rank == 0 && (issued & (1u << s)))
          mbar_wait_reset(&full[s], (issued_phase >> s) & 1u, status, kLimit, kWaitProducerDrain, s, false);
      if (ofs > 0) mbar_wait_reset(of_full, (ofs - 1) & 1, status, kLimit, kWaitProducerDrain, 0, false);
      if (*reinterpret_cast<volatile int *>(status + 1) != 0) {
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader), one thread
    if (rank == 0 && elect_one()) {
      const uint32_t base = smem_u32(smem);
      // K-major operands and M- / N-major ones
      const uint64_t desc_k = make_smem_desc(base, 16, 1024, kSwizzle128B);
      const uint64_t desc_mn = make_smem_desc(base, GP::kHalfBox, 1024, kSwizzle128B);
      int stage = 0, j = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (; ok && items.next(it, false); ++j) {
        const NsStage &s = g.stage[it.at % 3];
        const int n = tile_slots(s, it.c), blocks = (s.R + GP::kBK - 1) / GP::kBK;
        const int acc = j & 1;
        ok = mbar_wait_reset(&tmem_empty[acc], ((uint32_t)(j >> 1) & 1u) ^ 1u, status, kLimit, kWaitMmaTmemEmpty, it.at);
        if (!ok) break;
        tc_fence_after();
        if (g.inject_wait == 1 && j == 0 && !mbar_wait_reset(never, 0, status, kInjectedLimit, kWaitInjected, it.at)) break;
        const uint32_t idesc = make_idesc_f16(GP::kM, (uint32_t)n, s.a_mn, s.b_mn);
        const uint32_t d = tmem_base + (uint32_t)(acc * GP::kN);
        const uint64_t a_step = (s.a_mn ? 2048 : 32) >> 4, b_step = (s.b_mn ? 2048 : 32) >> 4;
        const uint64_t a_desc = s.a_mn ? desc_mn : desc_k, b_desc = (s.b_mn ? desc_mn : desc_k) + (GP::kATile >> 4);
        for (int kb = 0; kb < blocks; ++kb) {
          ok = mbar_wait_reset(&full[stage], phase, status, kLimit, kWaitMmaFull, kb);
          if (!ok) break;
          const uint64_t ad = a_desc + (uint64_t)((stage * L::kSlot) >> 4);
          const uint64_t bd = b_desc + (uint64_t)((stage * L::kSlot) >> 4);
          const int left = s.R - kb * GP::kBK;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (16 * kk < left) tc_mma_2sm_f16(d, ad + kk * a_step, bd + kk * b_step, idesc, kb > 0 || kk > 0 ? 1u : 0u);
          tc_commit_2sm(&empty[stage], 3);
          if (++stage == L::kStages) { stage = 0; phase ^= 1; }
        }
        if (ok) tc_commit_2sm(&tmem_full[acc], 3);
      }
      tc_commit_2sm(mma_done, 1);
      mbar_wait_reset(mma_done, 0, status, kLimit, kWaitMmaDone, 0, false);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ claims (leader), one thread
    if (rank == 0 && elect_one()) {
      const uint32_t ring1 = mapa_shared(smem_u32(ring), 1), full1 = mapa_shared(smem_u32(item_full), 1);
      int slot = 0;
      uint32_t phase = 0, wanted = 0;
      for (;;) {
        if (!mbar_wait_reset(item_empty + slot, phase ^ 1, status, kLimit, kWaitArrival, slot)) break;
        int4 v = ns_item(g, (int64_t)(uint32_t)atomicAdd(g.ticket, 1));
        // one look at the matrix's counter: if it is ready, the loads need not look (they are ordered after this one, through
        // the ring)
        if (v.w >= 0 && ld_acquire_gpu(g.done + v.x) >= ns_arrivals(g, v.w)) v.w |= kNsReady;
        ring[slot] = v;
        store_cluster_v4(ring1 + 16 * (uint32_t)slot, v);
        mbar_arrive(item_full + slot);
        mbar_arrive_cluster(full1 + 8 * (uint32_t)slot);
        if (v.w < 0) break;
        if (++slot == L::kClaims) { slot = 0; phase ^= 1; }
        // the next when this one's loads are nearly done: a pair that held one more would keep it from pairs that wait for
        // nothing (one matrix of 2048 x 2048 in 393 us instead of 242, of 512 x 512 in 132 instead of 90)
        if (!mbar_wait_reset(want, wanted, status, kLimit, kWaitArrival, slot)) break;
        wanted ^= 1;
      }
    }
    __syncwarp();
  } else if (warp >= GP::kFirstEpiWarp) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, ew = warp - GP::kFirstEpiWarp;
    unsigned char *buf = smem + L::kOffEpi + ew * L::kEpiBytes;
    uint32_t ofs = 0;
    for (int j = 0; items.next(it, true); ++j) {
      const int iteration = it.at / 3, k = it.at - 3 * iteration;
      const NsStage &s = g.stage[k];
      const CUtensorMap *d_map = k == 2 ? &maps.x32[(iteration + 1) & 1] : k == 1 || !g.square ? &maps.q32 : &maps.s32;
      const int acc = j & 1;
      // this warp's rows and columns of the tile: 128 columns, or 64 (of narrow tiles the first warps' alone)
      const int wide = s.tn > 128 ? 128 : 64, c_first = wide * (ew >> 2);
      const int row0 = it.m * GP::kM + (int)rank * 128 + 32 * q;
      const bool mirrored = s.symmetric && it.c * s.tn >= (it.m + 1) * GP::kM, in_rows = row0 + lane < s.M;
      float beta = s.beta, alpha = s.alpha;
      const float *of = reinterpret_cast<const float *>(smem + L::kOffOf);
      const bool of_rows = needs_of(it, s, k) && (k == 1 || g.wide), of_columns = k == 2 && !g.wide;
      if (of_rows || of_columns) {
        if (!__all_sync(0xffffffffu, mbar_wait_reset(of_full, ofs & 1, status, kLimit, kWaitEpiTmemFull, it.at))) break;
        ++ofs;
      }
      if (of_rows) {
        const float left = in_rows ? of[32 * q + lane] : 0.f;
        if (k == 1) beta += left; else alpha *= left;
        __syncwarp();
        if (lane == 0) mbar_arrive(of_empty);
      }
      if (!__all_sync(0xffffffffu, mbar_wait_reset(&tmem_full[acc], (uint32_t)(j >> 1) & 1u, status, kLimit,
                                                   kWaitEpiTmemFull, it.at)))
        break;
      tc_fence_after();
      const uint32_t t_row = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * GP::kN);
      bool kept = false;                                              // this warp wrote a part of a diagonal
      if (row0 < s.M) {
        for (int c0 = c_first; c0 < min(c_first + wide, s.tn); c0 += 64) {
          const int col0 = it.c * s.tn + c0;
          if (col0 >= s.C) break;
          uint32_t v[64];
#pragma unroll
          for (int h = 0; h < 64; h += 32)
            tmem_ld_32x32b_x32(t_row + (uint32_t)(c0 + h), *reinterpret_cast<uint32_t(*)[32]>(v + h));
          tmem_ld_wait();
          const int diagonal = row0 + lane - col0;                      // this lane's column on the diagonal
          uint32_t p[32];
          if (of_columns) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 f = *reinterpret_cast<const float2 *>(of + c0 + 2 * i);
              p[i] = pack_f16(alpha * f.x * __uint_as_float(v[2 * i]), alpha * f.y * __uint_as_float(v[2 * i + 1]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float x = fmaf(alpha, __uint_as_float(v[2 * i]), diagonal == 2 * i ? beta : 0.f);
              const float y = fmaf(alpha, __uint_as_float(v[2 * i + 1]), diagonal == 2 * i + 1 ? beta : 0.f);
              p[i] = pack_f16(x, y);
            }
          }
          if (k < 2 && !mirrored && col0 <= row0 && row0 < col0 + 64) {
            // the rows' part of the diagonal lies here
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 64; ++i) x = diagonal == i ? __uint_as_float(v[i]) : x;
            const bool of_square = k == 0 && g.square;
            if (in_rows)
              (of_square ? g.of_s : g.of_q)[(int64_t)it.e * g.ld_of + row0 + lane] =
                  left_of(fmaf(alpha, x, beta), of_square, g.stage[1].alpha);
            kept = true;
          }
          if (lane == 0) bulk_wait_read<0>();                          // the store before has read the staging
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(buf + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d_normal(d_map, buf, col0, row0, it.e);
            bulk_commit();
          }
          if (mirrored) {
            // the tile below the diagonal: lanes are columns there
            uint16_t *out = s.d + (int64_t)it.e * s.M * s.ld;
            const int col = row0 + 8 * (lane >> 3);
#pragma unroll
            for (int h = 0; h < 32; h += 16)
              turn_words<16>(p + h, lane, [&](int r, const uint4 &piece) {
                const int row = col0 + 2 * h + 8 * r + (lane & 7);
                if (row < s.C && col < s.M) *reinterpret_cast<uint4 *>(out + row * s.ld + col) = piece;
              });
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_done(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
      if (of_columns && lane == 0) mbar_arrive(of_empty);
      // published: this warp's part of the tile is in memory
      if (mirrored || kept) {
        fence_proxy_async_global();
        __threadfence();
        __syncwarp();
      }
      if (lane == 0) {
        bulk_wait<0>();
        fence_proxy_async_global();
        __threadfence();
        atomicAdd(g.done + it.e, 1);
      }
    }
    if (lane == 0) bulk_wait<0>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_2sm(tmem_base, 512);
  }
}

// ---------------------------------------------------------------- small matrices

// A matrix whose shorter side is at most 128 and whose other is at most 8 * 384: the whole
// call in one launch, momentum to update, a cluster of 1, 2, 4 or 8 CTAs for each matrix.
// The iterate X [n][k] lies in shared memory in FP16, cut along k over the
// cluster; S and Q [n][n] are in every CTA.  One copy of X serves as both operands
// of X X^T (summed along its rows) and as the right one of Q X (summed across
// them): the MMA reads either from the same 128-byte-swizzled blocks of 64
// columns.  Of X X^T each CTA has the part of its columns; it writes each row's part into
// the shared memory of the CTA that adds this row up in float32, which
// hands its rows of S to all (parts that are read from there instead: 75 instead of 60 us for 128 x 2048).  A stage is then an MMA of a few hundred
// nanoseconds, a commit and a pass from TMEM back to shared memory, where the
// kernel above needs a trip through L2 between any two: 4 us an iteration of 128 x 256
// instead of 10.
// What FP16 leaves of the diagonals costs 3 to 8 % of the time here (562 x 39: 7.5e-4 of the result instead of 3.3e-3, 128 x 384
// 7.5e-4 instead of 1.2e-3).
struct SmallArgs {
  Elementwise z;
  int n, k, kc;             // kc: columns of a CTA, a multiple of 64
  int steps, square;
  float gram_alpha, gram_beta, square_alpha, square_beta;
  int inject_wait;
};

struct SmallLayout {
  static constexpr int kMostN = 128, kMostColumns = 384, kThreads = 256;
  static constexpr int kBlock = kMostN * 128;                       // 64 columns of FP16
  static constexpr int kOffS = kMostColumns / 64 * kBlock, kOffQ = kOffS + 2 * kBlock;
  static constexpr int kOffPart = kOffQ + 2 * kBlock;               // [128][128] float32
  static constexpr int kOffBar = kOffPart + kMostN * kMostN * 4;
  static constexpr int kOffSums = kOffBar + 32;                     // 8 of this block's warps, 8 of the cluster's CTAs
  static constexpr int kOffDiag = kOffSums + 64;                    // [2][128] float32: of S, of Q
  static constexpr int kBytes = 1024 + kOffDiag + 2 * kMostN * 4;
};
static_assert(SmallLayout::kBytes <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void store_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}

// 16 bytes of columns col .. col + 7 of row r in blocks of 64 columns.
__device__ __forceinline__ int small_place(int r, int col) {
  return (col >> 6) * SmallLayout::kBlock + r * 128 + ((((col >> 3) & 7) ^ (r & 7)) << 4);
}

// Rows r .. r + 7 of X, columns col .. col + 7 of the matrix, of what is orthogonalised (0 past the matrix' ends), all
// loads before their use.  VEC 8: what is contiguous in memory in runs of 8, aligned to 16 bytes.
template <int VEC, bool WIDE>
__device__ __forceinline__ void small_values(const SmallArgs &g, int64_t base, int r, int col, float gs, bool fresh,
                                             float (&u)[8][8]) {
  float m[8][8];
#pragma unroll
  for (int a = 0; a < 8; ++a)
#pragma unroll
    for (int b = 0; b < 8; ++b) u[a][b] = m[a][b] = 0.f;
  // line a of the run's other direction, element b along the run
  auto at = [&](int a, int b) {
    return WIDE ? base + (int64_t)(r + a) * g.k + col + b : base + (int64_t)(col + a) * g.n + r + b;
  };
  auto inside = [&](int a, int b) { return WIDE ? r + a < g.n && col + b < g.k : r + b < g.n && col + a < g.k; };
#pragma unroll
  for (int a = 0; a < 8; ++a) {
    if (VEC == 8) {
      if (!inside(a, 0)) continue;
      load_values<8>(g.z.g, g.z.g_dtype, at(a, 0), u[a]);
      if (g.z.m) load_values<8>(g.z.m, MOE_F32, at(a, 0), m[a]);
    } else {
#pragma unroll
      for (int b = 0; b < 8; ++b)
        if (inside(a, b)) {
          float one[1];
          load_values<1>(g.z.g, g.z.g_dtype, at(a, b), one);
          u[a][b] = one[0];
          if (g.z.m) {
            load_values<1>(g.z.m, MOE_F32, at(a, b), one);
            m[a][b] = one[0];
          }
        }
    }
  }
  if (!g.z.m) return;
#pragma unroll
  for (int a = 0; a < 8; ++a) {
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const float d = g.z.gain * (u[a][b] * gs);
      if (fresh) m[a][b] = fmaf(g.z.mu, m[a][b], d);
      u[a][b] = g.z.nesterov ? fmaf(g.z.mu, m[a][b], d) : m[a][b];
    }
    if (!fresh) continue;
    if (VEC == 8) {
      if (inside(a, 0)) store_values<8>(g.z.m, MOE_F32, at(a, 0), m[a]);
    } else {
#pragma unroll
      for (int b = 0; b < 8; ++b)
        if (inside(a, b)) {
          const float one[1] = {m[a][b]};
          store_values<1>(g.z.m, MOE_F32, at(a, b), one);
        }
    }
  }
}

// WIDE: rows of X are rows in memory (else columns).
template <int VEC, bool WIDE>
__global__ void __launch_bounds__(SmallLayout::kThreads, 1) small_muon_kernel(const __grid_constant__ SmallArgs g) {
  using L = SmallLayout;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *sx = smem, *ss = smem + L::kOffS, *sq = smem + L::kOffQ, *part = smem + L::kOffPart;
  uint64_t *done = reinterpret_cast<uint64_t *>(smem + L::kOffBar), *never = done + 1;
  uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(done + 2);
  float *sums = reinterpret_cast<float *>(smem + L::kOffSums), *cluster_sums = sums + 8;
  float *of_s = reinterpret_cast<float *>(smem + L::kOffDiag), *of_q = of_s + L::kMostN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), ctas = (int)cluster_size();
  const int64_t e = blockIdx.x / ctas;
  int *status = g.z.status;
  if (warp == 0) {
    if (lane == 0) {
      mbar_init(done, 1);
      mbar_init(never, 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(tmem_ptr, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x < 16) status[threadIdx.x] = 0;
  const uint32_t tmem_base = *tmem_ptr, smem_base = smem_u32(smem);
  const int64_t base = e * (int64_t)g.n * g.k;
  const int first = rank * g.kc, across = g.kc / 8;            // this CTA's columns, eight at a time
  const float gs = g.z.grad_scale ? *g.z.grad_scale : 1.f;

  // Momentum and norm, blocks of 8 x 8 values; threads next to each other take what lies next to each other in memory.
  // A block's values are those of the same thread both times.
  const int down = (g.n + 7) / 8;
  auto block_at = [&](int i, int &r, int &c) {
    r = 8 * (WIDE ? i / across : i % down);
    c = 8 * (WIDE ? i % across : i / down);
  };
  float sum = 0.f;
  for (int i = threadIdx.x; i < down * across; i += L::kThreads) {
    int r, c;
    block_at(i, r, c);
    float u[8][8];
    small_values<VEC, WIDE>(g, base, r, first + c, gs, true, u);
#pragma unroll
    for (int j = 0; j < 64; ++j) sum = fmaf(u[j >> 3][j & 7], u[j >> 3][j & 7], sum);
  }
  sum = block_sum(sum, sums);
  if ((int)threadIdx.x < ctas) store_cluster_f32(mapa_shared(smem_u32(cluster_sums + rank), threadIdx.x), sum);
  if (threadIdx.x < 2 * L::kMostN) of_s[threadIdx.x] = 0.f;
  // rows past the last are zero
  for (int i = threadIdx.x; i < (L::kMostN - 8 * down) * across; i += L::kThreads)
    *reinterpret_cast<uint4 *>(sx + small_place(8 * down + i / across, 8 * (i % across))) = make_uint4(0, 0, 0, 0);
  cluster_sync();
  sum = 0.f;
  for (int c = 0; c < ctas; ++c) sum += cluster_sums[c];
  const float norm = sqrtf(sum), by = norm == 0.f ? 0.f : kScale / (norm < g.z.eps ? g.z.eps : norm);
  for (int i = threadIdx.x; i < down * across; i += L::kThreads) {
    int r, c;
    block_at(i, r, c);
    float u[8][8];
    small_values<VEC, WIDE>(g, base, r, first + c, gs, false, u);
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      uint32_t w[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        w[b] = WIDE ? pack_f16(u[a][2 * b] * by, u[a][2 * b + 1] * by) : pack_f16(u[2 * b][a] * by, u[2 * b + 1][a] * by);
      *reinterpret_cast<uint4 *>(sx + small_place(r + a, c)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }

  const int n16 = (g.n + 15) & ~15;
  const int share = (n16 + ctas - 1) / ctas;                    // rows of S that a CTA adds up
  // of S the rows that no CTA adds up, which no result depends on
  if (ctas > 1)
    for (int i = threadIdx.x; i < 2 * (L::kMostN - n16) * 8; i += L::kThreads) {
      const int at = (i & 1) * L::kBlock + (n16 * 8 + (i >> 1)) * 16;
      *reinterpret_cast<uint4 *>(ss + at) = *reinterpret_cast<uint4 *>(sq + at) = make_uint4(0, 0, 0, 0);
    }
  const uint32_t t_x = tmem_base + L::kMostN;                   // S and Q in columns 0 .. 127, X behind them
  uint32_t phase = 0;
  // what a stage writes is ordered before its MMAs, and these before what follows
  auto multiply = [&](auto issue) {
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && elect_one()) {
      tc_fence_after();
      issue();
      tc_commit(done);
    }
    __syncwarp();
    mbar_wait_reset(done, phase, status, kLimit, kWaitMmaDone, (int)phase);
    phase ^= 1;
    tc_fence_after();
  };
  // desc of an operand summed along its rows (K-major) or, X, across them
  auto desc_k = [&](int off) { return make_smem_desc(smem_base + (uint32_t)off, 16, 1024, kSwizzle128B); };
  const int q = warp & 3, row = 32 * q + lane;                  // this thread's TMEM lane: a row of S, Q and X
  const uint32_t t_lane = (uint32_t)(32 * q) << 16;
  auto left = [&](float x, bool of_square) { return left_of(x, of_square, g.square_alpha); };
  // S or Q from TMEM: factor, diagonal, FP16, into blocks at `to`
  auto take_square = [&](float alpha, float beta, unsigned char *to, float *diag, bool of_square) {
    uint32_t v[2][32];
    const int c1 = 32 * (warp >> 2);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (c1 + 64 * h < n16) tmem_ld_32x32b_x32(tmem_base + t_lane + (uint32_t)(c1 + 64 * h), v[h]);
    tmem_ld_wait();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c0 = c1 + 64 * h;
      if (c0 >= n16) break;
      const float add = c0 == 32 * q && row < g.n ? beta : 0.f;
      float mine = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + 8 * j + 2 * i;
          float x[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool on = 8 * j + 2 * i + k == lane;           // the diagonal, in the 32 columns from 32 q
            x[k] = c < n16 ? fmaf(alpha, __uint_as_float(v[h][8 * j + 2 * i + k]), on ? add : 0.f) : 0.f;
            if (on) mine = x[k];
          }
          w[i] = pack_f16(x[0], x[1]);
        }
        *reinterpret_cast<uint4 *>(to + small_place(row, c0 + 8 * j)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (c0 == 32 * q && row < g.n) diag[row] = left(mine, of_square);
    }
  };

  for (int it = 0; it < g.steps; ++it) {
    // S = X X^T + shift (without a square: Q)
    multiply([&] {
      if (g.inject_wait == 1 && it == 0) mbar_wait_reset(never, 0, status, kInjectedLimit, kWaitInjected, 0);
      const uint32_t idesc = make_idesc_f16(128, (uint32_t)n16, false, false);
      for (int b = 0; b < g.kc / 64; ++b) {
        const uint64_t d = desc_k(b * L::kBlock);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tmem_base, d + 2 * kk, d + 2 * kk, idesc, b > 0 || kk > 0 ? 1u : 0u);
      }
    });
    unsigned char *gram = g.square ? ss : sq;
    if (ctas == 1) {
      take_square(g.gram_alpha, g.gram_beta, gram, g.square ? of_s : of_q, g.square);
    } else {
      // this CTA's part of each row to the CTA that adds it up: [CTA][row of the share], 16 bytes at place c ^ (row & 7) of a
      // row's 32
      const int owner = row / share;
      const uint32_t to = mapa_shared(smem_u32(part) + (uint32_t)((rank * share + row - owner * share) * 512), (uint32_t)min(owner, ctas - 1));
      for (int c0 = 32 * (warp >> 2); c0 < n16; c0 += 64) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem_base + t_lane + (uint32_t)c0, v);
        tmem_ld_wait();
        if (row < n16)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int4 w = make_int4((int)v[4 * j], (int)v[4 * j + 1], (int)v[4 * j + 2], (int)v[4 * j + 3]);
            const int at = ((c0 / 4 + j) ^ (row & 7)) << 4;
            if (owner == rank)
              *reinterpret_cast<int4 *>(part + row * 512 + at) = w;      // its place is row
            else
              store_cluster_v4(to + (uint32_t)at, w);
          }
      }
      cluster_sync();
      for (int i = threadIdx.x; i < share * (n16 / 8); i += L::kThreads) {
        const int r = rank * share + i / (n16 / 8), c = i % (n16 / 8);
        if (r >= n16) break;
        float4 a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] = b[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < ctas) {
            const unsigned char *from = part + (k * share + i / (n16 / 8)) * 512;
            a[k] = *reinterpret_cast<const float4 *>(from + (((2 * c) ^ (r & 7)) << 4));
            b[k] = *reinterpret_cast<const float4 *>(from + (((2 * c + 1) ^ (r & 7)) << 4));
          }
        }
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          t[0] += a[k].x; t[1] += a[k].y; t[2] += a[k].z; t[3] += a[k].w;
          t[4] += b[k].x; t[5] += b[k].y; t[6] += b[k].z; t[7] += b[k].w;
        }
        float mine = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool on = 8 * c + j == r && r < g.n;
          t[j] = fmaf(g.gram_alpha, t[j], on ? g.gram_beta : 0.f);
          if (on) mine = t[j];
        }
        if (r >> 3 == c && r < g.n) {
          const float d = left(mine, g.square);
          float *at = (g.square ? of_s : of_q) + r;
          for (int k = 0; k < ctas; ++k) store_cluster_f32(mapa_shared(smem_u32(at), (uint32_t)k), d);
        }
        const int4 w = make_int4((int)pack_f16(t[0], t[1]), (int)pack_f16(t[2], t[3]), (int)pack_f16(t[4], t[5]), (int)pack_f16(t[6], t[7]));
        for (int k = 0; k < ctas; ++k)
          store_cluster_v4(mapa_shared(smem_u32(gram) + (uint32_t)small_place(r, 8 * c), (uint32_t)k), w);
      }
      cluster_sync();
    }
    if (g.square) {
      multiply([&] {
        const uint32_t idesc = make_idesc_f16(128, (uint32_t)n16, false, false);
        for (int kk = 0; 16 * kk < n16; ++kk) {
          const uint64_t d = desc_k(L::kOffS + (kk >> 2) * L::kBlock) + 2 * (kk & 3);
          tc_mma_f16(tmem_base, d, d, idesc, kk > 0 ? 1u : 0u);
        }
      });
      take_square(g.square_alpha, g.square_beta + of_s[row], sq, of_q, false);
    }
    // X = Q X
    multiply([&] {
      for (int c0 = 0; c0 < g.kc; c0 += 256) {
        const uint32_t idesc = make_idesc_f16(128, (uint32_t)min(256, g.kc - c0), false, true);
        const uint64_t x = make_smem_desc(smem_base + (uint32_t)(c0 / 64 * L::kBlock), L::kBlock, 1024, kSwizzle128B);
        for (int kk = 0; 16 * kk < n16; ++kk)
          tc_mma_f16(t_x + (uint32_t)c0, desc_k(L::kOffQ + (kk >> 2) * L::kBlock) + 2 * (kk & 3), x + 128 * kk, idesc, kk > 0 ? 1u : 0u);
      }
    });
    const float unit = of_q[row] / kScale;
    for (int c1 = 32 * (warp >> 2); c1 < g.kc; c1 += 128) {
      uint32_t v[2][32];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (c1 + 64 * h < g.kc) tmem_ld_32x32b_x32(t_x + t_lane + (uint32_t)(c1 + 64 * h), v[h]);
      tmem_ld_wait();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c0 = c1 + 64 * h;
        if (c0 >= g.kc) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_f16(unit * __uint_as_float(v[h][8 * j + 2 * i]), unit * __uint_as_float(v[h][8 * j + 2 * i + 1]));
          *reinterpret_cast<uint4 *>(sx + small_place(row, c0 + 8 * j)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  __syncthreads();

  // p = keep p - rate X, and its copy: runs of RUN values of memory, next to each other for threads next to each other
  constexpr int RUN = VEC;
  const float out = (g.z.update ? -g.z.rate : 1.f) * (1.f / kScale);
  const int mine = min(g.kc, g.k - first), lines = WIDE ? g.n : mine, runs = ((WIDE ? mine : g.n) + RUN - 1) / RUN;
#pragma unroll 4
  for (int i = threadIdx.x; i < lines * runs; i += L::kThreads) {
    const int line = i / runs, at_run = (i - line * runs) * RUN;
    const int64_t at = base + (WIDE ? (int64_t)line * g.k + first + at_run : (int64_t)(first + line) * g.n + at_run);
    float x[RUN], y[RUN];
    if (g.z.update) load_values<RUN>(g.z.p, g.z.p_dtype, at, y);
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      const int r = WIDE ? line : at_run + j, c = WIDE ? at_run + j : line;
      x[j] = __half2float(*reinterpret_cast<const __half *>(sx + small_place(r, c & ~7) + 2 * (c & 7)));
      y[j] = g.z.update ? fmaf(out, x[j], g.z.keep * y[j]) : out * x[j];
    }
    store_values<RUN>(g.z.p, g.z.p_dtype, at, y);
    if (g.z.copy) store_values<RUN>(g.z.copy, MOE_BF16, at, y);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// ---------------------------------------------------------------- host

struct Stack {              // of a call's workspace
  int64_t n, ldx, lds, ld_of;
  int parts;
  size_t sums, sync, x[2], s, q, of_s, of_q, total;
};

Stack stack_layout(int64_t E, int64_t N, int64_t K) {
  Stack w;
  w.n = std::min(N, K);
  // rows on whole lines of 128 bytes (8 matrices of 1000 x 520 in 145 us instead of 160, 12 of 600 x 1200 in 192 instead of
  // 214); on 16 bytes where that would be mostly padding
  auto pitch = [](int64_t columns) { return (int64_t)round_up(columns, columns > 64 ? 64 : 8); };
  w.ldx = pitch(K);
  w.lds = pitch(w.n);
  w.parts = (int)std::min<int64_t>(kMostParts, ceil_div(N * K, 4096));
  size_t off = kStatusBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round_up(bytes, 256);
    return at;
  };
  w.sums = take((size_t)E * w.parts * 4);
  w.sync = take((size_t)(E + 1) * 4);
  for (auto &x : w.x) x = take((size_t)E * N * w.ldx * 2);
  w.s = take((size_t)E * w.n * w.lds * 2);
  w.q = take((size_t)E * w.n * w.lds * 2);
  w.ld_of = (int64_t)round_up(w.n, 64);
  for (auto *of : {&w.of_s, &w.of_q}) *of = take(((size_t)E * w.ld_of + 256) * 4);       // (tiles read to their own ends)
  w.total = off;
  return w;
}

bool encode_f16(CUtensorMap *map, const void *base, int64_t cols, int64_t rows, int64_t E, int64_t ld, int box0, int box1) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)E};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(ld * rows) * 2};
  const cuuint32_t box[3] = {(cuuint32_t)box0, (cuuint32_t)box1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The width of a stage's tiles.  64 reduction values of a tile of 256, 128 or 64 columns keep a pair's tensor cores busy
// for 0.27, 0.14 or 0.07 us and bring 64, 48 or 40 KB to it, at 13.5 TB/s from L2 over all pairs that work and no more
// than 0.12 KB/ns for one SM; an item's start and end take some 3 us that the next one's loads do not hide in a chain of
// short stages, one more for the widest, whose warps drain twice the columns.  Of several matrices the next stage begins
// before a stage's last items are done.  Of the 27 choices for 21 stacks of 1 to 40 matrices of 200 to 3000 this one is
// within 4 % of the best.
void choose_tiles(NsStage &s, int64_t E) {
  const int64_t pairs = num_sms() / 2, mt = ceil_div(s.M, GP::kM);
  double best = 0;
  for (int tn : {256, 128, 64}) {
    const int64_t ct = ceil_div(s.C, tn), across = GP::kM / tn;
    int64_t items = 0;
    for (int64_t m = 0; m < mt; ++m) items += s.symmetric ? ct - m * across : ct;
    const double work = (double)std::min(pairs, E * items), kb = tn == 256 ? 64 : tn == 128 ? 48 : 40;
    const double block = std::max({0.27 * tn / 256, kb / 2 / 120, kb * work / 13.5e3});
    const double rounds = E == 1 ? (double)ceil_div(items, pairs) : std::max(1.0, (double)(E * items) / pairs);
    const double cost = rounds * (ceil_div(s.R, GP::kBK) * block + 0.5) + (tn == 256 ? 3.5 : 2.5);
    if (tn == 256 || cost < 0.97 * best) {
      best = cost;
      s.tn = tn;
      s.items = (int)items;
    }
  }
}

// The kernel's shared memory is allowed on the current device.
bool newton_schulz_ready() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(newton_schulz_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NsLayout::kBytes) != cudaSuccess)
      return false;
    ready.fetch_or(bit, std::memory_order_release);
  }
  return true;
}

int launch_newton_schulz(const NsMaps &maps, const NsArgs &g, cudaStream_t st) {
  int64_t most = 0;
  for (const NsStage &s : g.stage) most = std::max<int64_t>(most, (int64_t)g.E * s.items);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(num_sms() / 2, most)));
  cfg.blockDim = dim3(GP::kThreads);
  cfg.dynamicSmemBytes = NsLayout::kBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, newton_schulz_kernel, maps, g) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// The largest |a + b t + c t^2| of t in [0, 1], where the first iteration's Gram matrix has its eigenvalues: Q's entries are
// no larger, and its diagonal is a where the matrix has nothing.  FP16 with kScale ends at 15.99, and Q's own rounding is 2^-11 of that.
double largest_factor(const moe_newton_schulz &ns) {
  const double a = ns.a, b = ns.b, c = ns.c, t = c != 0.0 ? -b / (2.0 * c) : 0.0;
  const double inside = t > 0.0 && t < 1.0 ? std::fabs(a + t * (b + c * t)) : 0.0;
  return std::max({std::fabs(a), std::fabs(a + b + c), inside});
}

int check_stack(int64_t E, int64_t N, int64_t K, const moe_newton_schulz &ns, const int32_t *status, const void *workspace,
                size_t bytes) {
  if (E < 0 || N <= 0 || K <= 0 || ns.steps < 0 || ns.steps > 64) return MOE_ERR_INVALID_ARG;
  for (float f : {ns.a, ns.b, ns.c})
    if (!(std::fabs(f) <= 64.f)) return MOE_ERR_INVALID_ARG;
  if (!(ns.eps >= 0.f) || std::isinf(ns.eps) || (ns.c != 0.f && !(std::fabs(ns.b) <= 16.f * std::fabs(ns.c))))
    return MOE_ERR_INVALID_ARG;
  if (largest_factor(ns) > 15.9) return MOE_ERR_INVALID_ARG;
  if (N >= (1 << 20) || K >= (1 << 20) || E > 65535) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (E == 0) return MOE_OK;
  if (!workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(status, 4)) return MOE_ERR_MISALIGNED;
  return bytes < moe_muon_workspace_size(E, N, K) ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

// CTAs for a matrix of the small path, or 0: it is not one.  Matrices of one CTA in any number: 64 of 128 x 128 in 28 us, by
// the products' kernel 71, 200 of 64 x 256 in 53 and 95.  Clusters, whose exchange takes 4 of an iteration's 9 us, in as
// many rounds as pay: of two CTAs three (128 of 128 x 768 in 147 and 161, 200 of 40 x 600 in 103 and 182); of more, one, or two
// where n is at most 64 and the products' tiles are mostly empty (32 of 64 x 2048 in 109 and 122, 64 of 897 x 32 in 60 and
// 105; 20 of 128 x 2048 129 and 123, 64 of 64 x 2048, in four rounds, 183 and 173).
int small_cluster(int64_t E, int64_t N, int64_t K, const moe_newton_schulz &ns) {
  const int64_t n = std::min(N, K), k = std::max(N, K);
  if (n > SmallLayout::kMostN || k > 8 * SmallLayout::kMostColumns || ns.steps == 0) return 0;
  int ctas = 1;
  while (ceil_div(k, ctas) > SmallLayout::kMostColumns) ctas *= 2;
  const int rounds = ctas == 2 ? 3 : n <= 64 ? 2 : 1;
  return ctas == 1 || E * ctas <= rounds * num_sms() ? ctas : 0;
}

template <int VEC, bool WIDE>
int run_small(const Elementwise &z, const moe_newton_schulz &ns, int ctas, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(small_muon_kernel<VEC, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallLayout::kBytes) != cudaSuccess)
      return MOE_ERR_CUDA;
    ready.fetch_or(bit, std::memory_order_release);
  }
  SmallArgs g{};
  g.z = z;
  g.n = (int)std::min(z.N, z.K);
  g.k = (int)std::max(z.N, z.K);
  g.kc = (int)round_up(ceil_div(g.k, ctas), 64);
  g.steps = ns.steps;
  g.square = ns.c != 0.f;
  const float unit = 1.f / kScale, shift = g.square ? ns.b / (2.f * ns.c) : 0.f;
  g.gram_alpha = g.square ? unit : ns.b * unit;
  g.gram_beta = kScale * (g.square ? shift : ns.a);
  g.square_alpha = ns.c * unit;
  g.square_beta = kScale * (ns.a - ns.b * shift * 0.5f);
  g.inject_wait = injected_wait();
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(z.E * ctas));
  cfg.blockDim = dim3(SmallLayout::kThreads);
  cfg.dynamicSmemBytes = SmallLayout::kBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, small_muon_kernel<VEC, WIDE>, g) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// The stages of a stack's products and their tensor maps, and the kernel made ready: all that a call can be refused for, so that
// nothing is enqueued before.
int plan_newton_schulz(const Elementwise &z, const moe_newton_schulz &ns, const Stack &w, uint16_t *const (&x)[2], uint16_t *s,
                       uint16_t *q, NsMaps &maps, NsArgs &g) {
  const int64_t E = z.E, N = z.N, K = z.K;
  const bool wide = N <= K, square = ns.c != 0.f;                    // wide: the Gram matrix is that of the rows
  const float unit = 1.f / kScale, shift = square ? ns.b / (2.f * ns.c) : 0.f;
  const int n = (int)w.n, k = (int)std::max(N, K);
  g.stage[0] = {n, n, k, !wide, !wide, 1, 0, 0, square ? unit : ns.b * unit, kScale * (square ? shift : ns.a), square ? s : q, w.lds};
  g.stage[1] = {n, n, n, 0, 0, 1, 0, 0, ns.c * unit, kScale * (ns.a - ns.b * shift * 0.5f), q, w.lds};
  g.stage[2] = {(int)N, (int)K, n, 0, wide, 0, 0, 0, unit, 0.f, nullptr, 0};
  int64_t items = 0;                       // of a matrix, all iterations
  for (NsStage &stage : g.stage) {
    choose_tiles(stage, E);
    items += (int64_t)ns.steps * stage.items;
  }
  // Tickets (each pair draws one past the last) are 32 bits, a matrix's arrivals an int.  With up to 40 steps no stack that fits
  // 288 GB reaches either: 12 bytes a value, 256 values a tile at the least in stacks that long.
  if (E * items + num_sms() > 0xffffffffLL || 2 * GP::kEpiWarps * items > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED_SHAPE;
  bool ok = true;
  for (int i = 0; i < 2; ++i)
    ok = ok && encode_f16(&maps.x128[i], x[i], K, N, E, w.ldx, GP::kBK, 128) && encode_f16(&maps.x32[i], x[i], K, N, E, w.ldx, 64, 32) &&
         encode_f16(&maps.x64[i], x[i], K, N, E, w.ldx, 64, 64);
  ok = ok && encode_f16(&maps.s128, s, n, n, E, w.lds, GP::kBK, 128) && encode_f16(&maps.s32, s, n, n, E, w.lds, 64, 32) &&
       encode_f16(&maps.q128, q, n, n, E, w.lds, GP::kBK, 128) && encode_f16(&maps.q32, q, n, n, E, w.lds, 64, 32);
  if (!ok || !newton_schulz_ready()) return MOE_ERR_CUDA;
  g.E = (int)E;
  g.steps = ns.steps;
  g.wide = wide;
  g.square = square;
  g.ticket = z.sync;
  g.done = z.sync + 1;
  g.ld_of = (int)w.ld_of;
  g.inject_wait = injected_wait();
  g.status = z.status;
  return MOE_OK;
}

template <int VEC>
int run_stack(Elementwise z, const moe_newton_schulz &ns, const Stack &w, char *base, cudaStream_t st) {
  z.parts = w.parts;
  z.per = (int)round_up(ceil_div(z.N * z.K, z.parts), 8 * 256);
  z.ld = w.ldx;
  z.sums = reinterpret_cast<float *>(base + w.sums);
  z.sync = reinterpret_cast<int *>(base + w.sync);
  uint16_t *const x[2] = {reinterpret_cast<uint16_t *>(base + w.x[0]), reinterpret_cast<uint16_t *>(base + w.x[1])};
  uint16_t *s = reinterpret_cast<uint16_t *>(base + w.s), *q = reinterpret_cast<uint16_t *>(base + w.q);
  NsMaps maps;
  NsArgs g{};
  g.of_s = reinterpret_cast<float *>(base + w.of_s);
  g.of_q = reinterpret_cast<float *>(base + w.of_q);
  int rc = ns.steps > 0 ? plan_newton_schulz(z, ns, w, x, s, q, maps, g) : MOE_OK;
  if (rc != MOE_OK) return rc;
  z.x = x[0];
  const dim3 grid((unsigned)z.parts, (unsigned)z.E), block(256);
  rc = launch_pdl(momentum_kernel<VEC>, grid, block, 0, st, z);
  if (rc == MOE_OK) rc = launch_pdl(scale_kernel<VEC>, grid, block, 0, st, z);
  if (rc == MOE_OK && ns.steps > 0) rc = launch_newton_schulz(maps, g, st);
  if (rc != MOE_OK) return rc;
  z.x = x[ns.steps & 1];
  return launch_pdl(update_kernel<VEC>, grid, block, 0, st, z);
}

int run_stack(const Elementwise &z, const moe_newton_schulz &ns, void *workspace, cudaStream_t st) {
  const Stack w = stack_layout(z.E, z.N, z.K);
  const bool vec = z.K % 8 == 0 && aligned(z.g, 16) && aligned(z.m, 16) && aligned(z.p, 16) && aligned(z.copy, 16);
  if (const int ctas = small_cluster(z.E, z.N, z.K, ns))
    return z.N <= z.K ? (vec ? run_small<8, true>(z, ns, ctas, st) : run_small<1, true>(z, ns, ctas, st))
                      : (vec ? run_small<8, false>(z, ns, ctas, st) : run_small<1, false>(z, ns, ctas, st));
  return vec ? run_stack<8>(z, ns, w, static_cast<char *>(workspace), st)
             : run_stack<1>(z, ns, w, static_cast<char *>(workspace), st);
}

bool dtype_valid(int32_t d) { return d == MOE_BF16 || d == MOE_F32; }

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" size_t moe_muon_workspace_size(int64_t E, int64_t N, int64_t K) {
  if (E < 0 || N <= 0 || K <= 0 || E > 65535 || N >= (1 << 20) || K >= (1 << 20)) return 0;
  return stack_layout(E, N, K).total;
}

extern "C" int moe_orthogonalize(const moe_orthogonalize_args *a, cudaStream_t stream) {
  if (!a || a->struct_size != sizeof(moe_orthogonalize_args) || !dtype_valid(a->x_dtype) || !dtype_valid(a->out_dtype))
    return MOE_ERR_INVALID_ARG;
  const int rc = check_stack(a->E, a->N, a->K, a->ns, a->status, a->workspace, a->workspace_bytes);
  if (rc != MOE_OK || a->E == 0) return rc;
  if (!a->x || !a->out) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->x, a->x_dtype == MOE_F32 ? 4 : 2) || !aligned(a->out, a->out_dtype == MOE_F32 ? 4 : 2))
    return MOE_ERR_MISALIGNED;
  Elementwise z{};
  z.E = a->E;
  z.N = a->N;
  z.K = a->K;
  z.g = a->x;
  z.g_dtype = a->x_dtype;
  z.eps = a->ns.eps;
  z.status = a->status ? a->status : reinterpret_cast<int *>(a->workspace);
  z.p = a->out;
  z.p_dtype = a->out_dtype;
  z.update = 0;
  return run_stack(z, a->ns, a->workspace, stream);
}

extern "C" int moe_muon_step(const moe_muon_args *a, cudaStream_t stream) {
  if (!a || a->struct_size != sizeof(moe_muon_args) || !dtype_valid(a->p_dtype) || !dtype_valid(a->g_dtype) ||
      (a->nesterov != 0 && a->nesterov != 1))
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(a->lr) || !std::isfinite(a->weight_decay) || !std::isfinite(a->scale) || !(a->momentum >= 0.0) ||
      !(a->momentum < 1.0))
    return MOE_ERR_INVALID_ARG;
  const int rc = check_stack(a->E, a->N, a->K, a->ns, a->status, a->workspace, a->workspace_bytes);
  if (rc != MOE_OK || a->E == 0) return rc;
  if (!a->p || !a->g || !a->m) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->p, a->p_dtype == MOE_F32 ? 4 : 2) || !aligned(a->g, a->g_dtype == MOE_F32 ? 4 : 2) || !aligned(a->m, 4) ||
      !aligned(a->copy, 2) || !aligned(a->grad_scale, 4))
    return MOE_ERR_MISALIGNED;
  Elementwise z{};
  z.E = a->E;
  z.N = a->N;
  z.K = a->K;
  z.g = a->g;
  z.g_dtype = a->g_dtype;
  z.m = a->m;
  z.grad_scale = a->grad_scale;
  z.mu = (float)a->momentum;
  z.gain = (float)(1.0 - a->momentum);
  z.nesterov = a->nesterov;
  z.eps = a->ns.eps;
  z.status = a->status ? a->status : reinterpret_cast<int *>(a->workspace);
  z.p = a->p;
  z.p_dtype = a->p_dtype;
  z.copy = a->copy;
  z.update = 1;
  z.keep = (float)(1.0 - a->lr * a->weight_decay);
  z.rate = (float)(a->lr * a->scale);
  return run_stack(z, a->ns, a->workspace, stream);
}
