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
  const int64_t e = blockIdx.y, size = z.N * z.K;
  float sum = 0.f;
  for (int i = threadIdx.x; i < z.parts; i += 256) sum += z.sums[e * z.parts + i];
  sum = block_sum(sum, red);
  // (max written so that a NaN stays one)
  const float norm = sqrtf(sum), by = norm == 0.f ? 0.f : kScale / (norm < z.eps ? z.eps : norm);
  const float gs = z.grad_scale ? *z.grad_scale : 1.f;
  const int64_t i0 = (int64_t)blockIdx.x * z.per, i1 = min(i0 + z.per, size);
#pragma unroll 2
  for (int64_t i = i0 + threadIdx.x * VEC; i < i1; i += 256 * VEC) {
    float u[VEC];
    values_of<VEC>(z, e * size + i, gs, false, u);
    if (VEC == 8) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) w[k] = pack_f16(u[2 * k] * by, u[2 * k + 1] * by);
      *reinterpret_cast<uint4 *>(z.x + e * size + i) = make_uint4(w[0], w[1], w[2], w[3]);      // ld is K
    } else {
      const int64_t r = i / z.K;
      reinterpret_cast<__half *>(z.x)[(e * z.N + r) * z.ld + (i - r * z.K)] = __float2half_rn(u[0] * by);
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
      const uint4 q = *reinterpret_cast<const uint4 *>(z.x + e * size + i);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    } else {
      const int64_t r = i / z.K;
      x[0] = __half2float(reinterpret_cast<const __half *>(z.x)[(e * z.N + r) * z.ld + (i - r * z.K)]);
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

// D[e] = alpha A[e] B[e]^T + beta on the diagonal, FP16, for a stack: M rows, C
// columns, sums over R.  Pairs of CTAs (M = 256, N = 256 per item), as
// grouped_kernel.cuh's weights' gradient: 64 reduction values a stage, two
// accumulators, boxes of 32 rows x 128 bytes through TMA.
struct ProductArgs {
  int E, M, C, R;
  int symmetric;            // D is: tiles on and above the diagonal, each stored twice
  float alpha, beta;
  uint16_t *d;
  int64_t ld, stride;       // of d, for the tiles below the diagonal
  int inject_wait;
  int *status;
};

struct ProductMaps {
  CUtensorMap a, b, d;
};

struct PL {
  static constexpr int kStages = 6, kSlot = 32768, kEpiBytes = 4096;
  static constexpr int kOffEpi = kStages * kSlot;
  static constexpr int kOffBar = kOffEpi + GP::kEpiWarps * kEpiBytes;
  static constexpr int kNumBars = 2 * kStages + 6;
  static constexpr int kOffTmemPtr = (kOffBar + 8 * kNumBars + 63) & ~63;
  static constexpr int kBytes = 1024 + kOffTmemPtr + 64;
};
static_assert(PL::kBytes <= 232448, "shared memory of one CTA");

struct Tile {
  int e, m, c, n;           // N slots (a multiple of 32)
};

__device__ __forceinline__ Tile tile_at(const ProductArgs &g, int w, int per, int mt, int ct) {
  Tile t;
  t.e = w / per;
  int i = w - t.e * per;
  if (g.symmetric) {
    t.m = 0;
    while (i >= mt - t.m) {
      i -= mt - t.m;
      ++t.m;
    }
    t.c = t.m + i;
  } else {
    t.m = i / ct;
    t.c = i - t.m * ct;
  }
  t.n = min(GP::kN, (g.C - t.c * GP::kN + 31) & ~31);
  return t;
}

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

// AMN / BMN: the operand's M (N) index is the contiguous one in memory.
template <bool AMN, bool BMN>
__global__ void __launch_bounds__(GP::kThreads, 1) product_kernel(const __grid_constant__ ProductMaps maps,
                                                                  const ProductArgs g) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + PL::kOffBar);     // leader: both CTAs' copies of a stage
  uint64_t *empty = full + PL::kStages;                                  // each CTA: stage consumed
  uint64_t *tmem_full = empty + PL::kStages;                             // each CTA: accumulator ready
  uint64_t *tmem_empty = tmem_full + 2;                                  // leader: both CTAs drained it
  uint64_t *mma_done = tmem_empty + 2;
  uint64_t *never = mma_done + 1;
  uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(smem + PL::kOffTmemPtr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;
  int *status = g.status;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.a);
      tma_prefetch_desc(&maps.b);
      tma_prefetch_desc(&maps.d);
    }
  } else if (warp == 2) {
    if (lane == 0) {
      for (int s = 0; s < PL::kStages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      for (int a = 0; a < 2; ++a) {
        mbar_init(&tmem_full[a], 1);
        mbar_init(&tmem_empty[a], 2 * GP::kEpiWarps);
      }
      mbar_init(mma_done, 1);
      mbar_init(never, 1);
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
  const int mt = (g.M + GP::kM - 1) / GP::kM, ct = (g.C + GP::kN - 1) / GP::kN;
  const int per = g.symmetric ? mt * (mt + 1) / 2 : mt * ct;
  const int total = g.E * per, blocks = (g.R + GP::kBK - 1) / GP::kBK;

  if (warp == 0) {
    // ------------------------------------------------------------ loads (both CTAs), one thread
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      const uint32_t full0 = mapa_shared(smem_u32(full), 0);
      const uint64_t policy = l2_policy(false);
      fence_proxy_async_global();       // what the kernel before stored from registers is read by TMA
      for (int w = cluster; w < total && ok; w += step) {
        const Tile t = tile_at(g, w, per, mt, ct);
        const int row = t.m * GP::kM + (int)rank * 128, col = t.c * GP::kN + (int)rank * (t.n >> 1);
        for (int kb = 0; kb < blocks; ++kb) {
          unsigned char *a = smem + stage * PL::kSlot, *b = a + GP::kATile;
          const uint32_t bar = full0 + 8 * (uint32_t)stage;
          const int k0 = kb * GP::kBK;
          if (!mbar_wait_reset(&empty[stage], phase ^ 1, status, kLimit, kWaitProducerEmpty, kb)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * PL::kSlot);
          if (AMN) {
#pragma unroll
            for (int j = 0; j < 2; ++j) tma_load_3d_2sm(a + j * GP::kHalfBox, &maps.a, bar, row + 64 * j, k0, t.e, policy);
          } else {
            tma_load_3d_2sm(a, &maps.a, bar, k0, row, t.e, policy);
          }
          if (BMN) {
#pragma unroll
            for (int j = 0; j < 2; ++j) tma_load_3d_2sm(b + j * GP::kHalfBox, &maps.b, bar, col + 64 * j, k0, t.e, policy);
          } else {
            tma_load_3d_2sm(b, &maps.b, bar, k0, col, t.e, policy);
          }
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == PL::kStages) { stage = 0; phase ^= 1; }
        }
      }
      // no CTA leaves with copies in flight (as in grouped_kernel)
      for (int s = 0; s < PL::kStages; ++s)
        if (rank == 0 && (issued & (1u << s)))
          mbar_wait_reset(&full[s], (issued_phase >> s) & 1u, status, kLimit, kWaitProducerDrain, s, false);
      if (*reinterpret_cast<volatile int *>(status + 1) != 0) {
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader), one thread
    if (rank == 0 && elect_one()) {
      constexpr uint64_t kAStep = (AMN ? 2048 : 32) >> 4, kBStep = (BMN ? 2048 : 32) >> 4;
      const uint64_t a_desc = make_smem_desc(smem_u32(smem), AMN ? GP::kHalfBox : 16, 1024, kSwizzle128B);
      const uint64_t b_desc = make_smem_desc(smem_u32(smem) + GP::kATile, BMN ? GP::kHalfBox : 16, 1024, kSwizzle128B);
      int stage = 0, j = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int w = cluster; w < total && ok; w += step, ++j) {
        const Tile t = tile_at(g, w, per, mt, ct);
        const int acc = j & 1;
        if (!mbar_wait_reset(&tmem_empty[acc], ((uint32_t)(j >> 1) & 1u) ^ 1u, status, kLimit, kWaitMmaTmemEmpty, w)) break;
        tc_fence_after();
        if (g.inject_wait == 1 && j == 0 && !mbar_wait_reset(never, 0, status, kInjectedLimit, kWaitInjected, w)) break;
        const uint32_t idesc = make_idesc_f16(GP::kM, (uint32_t)t.n, AMN, BMN);
        const uint32_t d = tmem_base + (uint32_t)(acc * GP::kN);
        for (int kb = 0; kb < blocks; ++kb) {
          if (!mbar_wait_reset(&full[stage], phase, status, kLimit, kWaitMmaFull, kb)) {
            ok = false;
            break;
          }
          const uint64_t ad = a_desc + (uint64_t)((stage * PL::kSlot) >> 4);
          const uint64_t bd = b_desc + (uint64_t)((stage * PL::kSlot) >> 4);
          const int left = g.R - kb * GP::kBK;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (16 * kk < left) tc_mma_2sm_f16(d, ad + kk * kAStep, bd + kk * kBStep, idesc, kb > 0 || kk > 0 ? 1u : 0u);
          tc_commit_2sm(&empty[stage], 3);
          if (++stage == PL::kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        tc_commit_2sm(&tmem_full[acc], 3);
      }
      tc_commit_2sm(mma_done, 1);
      mbar_wait_reset(mma_done, 0, status, kLimit, kWaitMmaDone, 0, false);
    }
    __syncwarp();
  } else if (warp >= GP::kFirstEpiWarp) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, ew = warp - GP::kFirstEpiWarp;
    unsigned char *buf = smem + PL::kOffEpi + ew * PL::kEpiBytes;
    int j = 0;
    for (int w = cluster; w < total; w += step, ++j) {
      const Tile t = tile_at(g, w, per, mt, ct);
      const int acc = j & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_reset(&tmem_full[acc], (uint32_t)(j >> 1) & 1u, status, kLimit,
                                                   kWaitEpiTmemFull, w)))
        break;
      tc_fence_after();
      const int row0 = t.m * GP::kM + (int)rank * 128 + 32 * q, col0 = t.c * GP::kN + 128 * (ew >> 2);
      const uint32_t t_row = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * GP::kN + 128 * (ew >> 2));
      if (row0 < g.M) {
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 64) {
          if (col0 + c0 >= g.C) break;
          uint32_t v[64];
#pragma unroll
          for (int h = 0; h < 64; h += 32)
            tmem_ld_32x32b_x32(t_row + (uint32_t)(c0 + h), *reinterpret_cast<uint32_t(*)[32]>(v + h));
          tmem_ld_wait();
          const int diagonal = row0 + lane - (col0 + c0);               // this lane's column on the diagonal
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float x = fmaf(g.alpha, __uint_as_float(v[2 * i]), diagonal == 2 * i ? g.beta : 0.f);
            const float y = fmaf(g.alpha, __uint_as_float(v[2 * i + 1]), diagonal == 2 * i + 1 ? g.beta : 0.f);
            p[i] = pack_f16(x, y);
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
            tma_store_3d_normal(&maps.d, buf, col0 + c0, row0, t.e);
            bulk_commit();
          }
          if (g.symmetric && t.c > t.m) {
            // the tile below the diagonal: lanes are columns there
            uint16_t *out = g.d + t.e * g.stride;
            const int col = row0 + 8 * (lane >> 3);
#pragma unroll
            for (int h = 0; h < 32; h += 16)
              turn_words<16>(p + h, lane, [&](int r, const uint4 &piece) {
                const int row = col0 + c0 + 2 * h + 8 * r + (lane & 7);
                if (row < g.C && col < g.M) *reinterpret_cast<uint4 *>(out + row * g.ld + col) = piece;
              });
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_done(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
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

// ---------------------------------------------------------------- host

struct Stack {              // of a call's workspace
  int64_t n, ldx, lds;
  int parts;
  size_t sums, x[2], s, q, total;
};

Stack stack_layout(int64_t E, int64_t N, int64_t K) {
  Stack w;
  w.n = std::min(N, K);
  w.ldx = (int64_t)round_up(K, 8);
  w.lds = (int64_t)round_up(w.n, 8);
  w.parts = (int)std::min<int64_t>(kMostParts, ceil_div(N * K, 4096));
  size_t off = kStatusBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round_up(bytes, 256);
    return at;
  };
  w.sums = take((size_t)E * w.parts * 4);
  for (auto &x : w.x) x = take((size_t)E * N * w.ldx * 2);
  w.s = take((size_t)E * w.n * w.lds * 2);
  w.q = take((size_t)E * w.n * w.lds * 2);
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

// a [M rows of R, or R rows of M], b [C rows of R, or R rows of C], d [M][C].
template <bool AMN, bool BMN>
int launch_product(const uint16_t *a, int64_t lda, const uint16_t *b, int64_t ldb, uint16_t *d, int64_t ldd, int64_t E,
                   int64_t M, int64_t C, int64_t R, bool symmetric, float alpha, float beta, int *status, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(product_kernel<AMN, BMN>, cudaFuncAttributeMaxDynamicSharedMemorySize, PL::kBytes) != cudaSuccess)
      return MOE_ERR_CUDA;
    ready.fetch_or(bit, std::memory_order_release);
  }
  ProductMaps maps;
  const bool ok = (AMN ? encode_f16(&maps.a, a, M, R, E, lda, 64, GP::kBK) : encode_f16(&maps.a, a, R, M, E, lda, GP::kBK, 128)) &&
                  (BMN ? encode_f16(&maps.b, b, C, R, E, ldb, 64, GP::kBK) : encode_f16(&maps.b, b, R, C, E, ldb, GP::kBK, 128)) &&
                  encode_f16(&maps.d, d, C, M, E, ldd, 64, 32);
  if (!ok) return MOE_ERR_CUDA;
  const int64_t mt = ceil_div(M, GP::kM), items = E * (symmetric ? mt * (mt + 1) / 2 : mt * ceil_div(C, GP::kN));
  if (items > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED_SHAPE;
  const ProductArgs g{(int)E, (int)M, (int)C, (int)R, symmetric, alpha, beta, d, ldd, M * ldd, injected_wait(), status};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(num_sms() / 2, items)));
  cfg.blockDim = dim3(GP::kThreads);
  cfg.dynamicSmemBytes = PL::kBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, product_kernel<AMN, BMN>, maps, g) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int check_stack(int64_t E, int64_t N, int64_t K, const moe_newton_schulz &ns, const int32_t *status, const void *workspace,
                size_t bytes) {
  if (E < 0 || N <= 0 || K <= 0 || ns.steps < 0 || ns.steps > 64) return MOE_ERR_INVALID_ARG;
  for (float f : {ns.a, ns.b, ns.c})
    if (!(std::fabs(f) <= 64.f)) return MOE_ERR_INVALID_ARG;
  if (!(ns.eps >= 0.f) || std::isinf(ns.eps) || (ns.c != 0.f && !(std::fabs(ns.b) <= 16.f * std::fabs(ns.c))))
    return MOE_ERR_INVALID_ARG;
  if (N >= (1 << 20) || K >= (1 << 20) || E > 65535) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (E == 0) return MOE_OK;
  if (!workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(status, 4)) return MOE_ERR_MISALIGNED;
  return bytes < moe_muon_workspace_size(E, N, K) ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

template <int VEC>
int run_stack(Elementwise z, const moe_newton_schulz &ns, const Stack &w, char *base, cudaStream_t st) {
  const int64_t E = z.E, N = z.N, K = z.K;
  z.parts = w.parts;
  z.per = (int)round_up(ceil_div(N * K, z.parts), 8 * 256);
  z.ld = w.ldx;
  z.sums = reinterpret_cast<float *>(base + w.sums);
  uint16_t *x[2] = {reinterpret_cast<uint16_t *>(base + w.x[0]), reinterpret_cast<uint16_t *>(base + w.x[1])};
  uint16_t *s = reinterpret_cast<uint16_t *>(base + w.s), *q = reinterpret_cast<uint16_t *>(base + w.q);
  z.x = x[0];
  const dim3 grid((unsigned)z.parts, (unsigned)E), block(256);
  int rc = launch_pdl(momentum_kernel<VEC>, grid, block, 0, st, z);
  if (rc == MOE_OK) rc = launch_pdl(scale_kernel<VEC>, grid, block, 0, st, z);
  const bool wide = N <= K;                 // the Gram matrix is that of the rows
  const float unit = 1.f / kScale, shift = ns.c != 0.f ? ns.b / (2.f * ns.c) : 0.f;
  const int64_t n = w.n, k = std::max(N, K);
  for (int i = 0; i < ns.steps && rc == MOE_OK; ++i) {
    const uint16_t *from = x[i & 1];
    uint16_t *to = x[(i + 1) & 1], *gram = ns.c != 0.f ? s : q;
    const float alpha = ns.c != 0.f ? unit : ns.b * unit, beta = kScale * (ns.c != 0.f ? shift : ns.a);
    rc = wide ? launch_product<false, false>(from, w.ldx, from, w.ldx, gram, w.lds, E, n, n, k, true, alpha, beta, z.status, st)
              : launch_product<true, true>(from, w.ldx, from, w.ldx, gram, w.lds, E, n, n, k, true, alpha, beta, z.status, st);
    if (rc == MOE_OK && ns.c != 0.f)
      rc = launch_product<false, false>(s, w.lds, s, w.lds, q, w.lds, E, n, n, n, true, ns.c * unit,
                                        kScale * (ns.a - ns.b * shift * 0.5f), z.status, st);
    if (rc == MOE_OK)
      rc = wide ? launch_product<false, true>(q, w.lds, from, w.ldx, to, w.ldx, E, N, K, n, false, unit, 0.f, z.status, st)
                : launch_product<false, false>(from, w.ldx, q, w.lds, to, w.ldx, E, N, K, n, false, unit, 0.f, z.status, st);
  }
  if (rc != MOE_OK) return rc;
  z.x = x[ns.steps & 1];
  return launch_pdl(update_kernel<VEC>, grid, block, 0, st, z);
}

int run_stack(const Elementwise &z, const moe_newton_schulz &ns, void *workspace, cudaStream_t st) {
  const Stack w = stack_layout(z.E, z.N, z.K);
  const bool vec = z.K % 8 == 0 && aligned(z.g, 16) && aligned(z.m, 16) && aligned(z.p, 16) && aligned(z.copy, 16);
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
