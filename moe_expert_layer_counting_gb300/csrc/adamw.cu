// adamw.cu -- one AdamW step over many tensors (include/moe_adamw.h has the
// formulas and the 8-bit states' format).
//
// Bound by HBM: 28 bytes a value with float32 states (p read and written, BF16
// gradient and copy, m and v read and written), 16.1 with 8-bit states.  The
// table of tensors travels in the kernel's parameters (no copy to the device,
// nothing kept between calls), up to kMany per launch; a block finds its
// tensor by bisection of the tensors' first blocks.  A thread owns 8
// consecutive values, four neighbours a 32-value group of the 8-bit states.
// Measured: float32 states, 201 M values in 805 us (7.0 TB/s); 8-bit states,
// 352 M values in 818 us (6.9 TB/s; 837 as 19 tensors).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "../../include/moe_adamw.h"
#include "host_common.h"
#include "ptx.cuh"

namespace mxq {

namespace {

// Threads of a block.  With 8-bit states the arithmetic of one warp hides less
// behind the others' loads, and blocks that come and go one by one keep the
// warps of an SM apart: 352 M values in 818 us with 64 threads, 822 with 128, 843
// with 256, 1105 with 512; float32 states 1403, 1403, 1394 and 1400.
template <bool kSmall> constexpr int kThreads = kSmall ? 64 : 256;
constexpr int kRounds = 2;                                   // vectors per thread
template <bool kSmall> constexpr int64_t kChunk = (int64_t)kThreads<kSmall> * 8 * kRounds;      // values per block

struct AdamEntry {
  int64_t n;
  void *p;
  const void *g;
  void *m, *v;
  uint8_t *ms, *vs;
  uint16_t *copy;
};

template <int TENSORS>
struct AdamTable {
  AdamEntry t[TENSORS];
  int first[TENSORS + 1];          // first block of each tensor
  int count;
  float beta1, one_minus_beta1, beta2, one_minus_beta2, keep, rate, root_scale, eps;
  const float *grad_scale;
};

struct V8 {
  float v[8];
};

// Eight values as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ V8 get() const { return V8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
template <> struct Raw8<uint16_t> {
  uint4 q;
  __device__ __forceinline__ V8 get() const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[2 * i] = bf16_bits_to_float(w[i] & 0xFFFFu);
      r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    return r;
  }
};
// `live` (1 .. 8) of them; the others read as zero.
__device__ __forceinline__ Raw8<float> load_raw(const float *p, int live) {
  Raw8<float> r;
  if (live == 8) {
    r.a = reinterpret_cast<const float4 *>(p)[0];
    r.b = reinterpret_cast<const float4 *>(p)[1];
  } else {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < live ? p[j] : 0.f;
    r.a = make_float4(f[0], f[1], f[2], f[3]);
    r.b = make_float4(f[4], f[5], f[6], f[7]);
  }
  return r;
}
__device__ __forceinline__ Raw8<uint16_t> load_raw(const uint16_t *p, int live) {
  Raw8<uint16_t> r;
  if (live == 8) {
    r.q = *reinterpret_cast<const uint4 *>(p);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (2 * i < live ? p[2 * i] : 0u) | (2 * i + 1 < live ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    r.q = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}
__device__ __forceinline__ uint16_t to_bf16(float f) {
  const __nv_bfloat16 b = __float2bfloat16_rn(f);
  return *reinterpret_cast<const uint16_t *>(&b);
}
__device__ __forceinline__ void put(float *p, float f) { *p = f; }
__device__ __forceinline__ void put(uint16_t *p, float f) { *p = to_bf16(f); }
__device__ __forceinline__ void store8(float *p, const V8 &f) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}
__device__ __forceinline__ void store8(uint16_t *p, const V8 &f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)to_bf16(f.v[2 * i]) | ((uint32_t)to_bf16(f.v[2 * i + 1]) << 16);
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// `live` (1 .. 8) of 8 values.
template <typename T>
__device__ __forceinline__ void store_some(T *p, const V8 &f, int live) {
  if (live == 8) {
    store8(p, f);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < live) put(p + j, f.v[j]);
}
__device__ __forceinline__ uint2 load_codes(const uint8_t *p, int live) {
  if (live == 8) return *reinterpret_cast<const uint2 *>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < live) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t *p, const uint2 &c, int live) {
  if (live == 8) {
    *reinterpret_cast<uint2 *>(p) = c;
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < live) p[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
}

// 2^(byte - 127) (byte 0: a float32 subnormal).
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

__device__ __forceinline__ V8 decode8(const uint2 &c, uint32_t byte) {
  const float s = scale_of(byte);
  const uint32_t w[2] = {c.x, c.y};
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t two = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    r.v[2 * i] = f.x * s;
    r.v[2 * i + 1] = f.y * s;
  }
  return r;
}

// The largest of four lanes' values (a group's 32).
__device__ __forceinline__ float group_max(float a) {
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  return fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
}

// Codes of eight values under the scale 2^e.
__device__ __forceinline__ uint2 encode8(const V8 &f, int e) {
  const float inv = pow2_neg(e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = cvt_e4m3x2(f.v[2 * i] * inv, f.v[2 * i + 1] * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Within 2 units in the last place; FTZ: a subnormal's root is 0.
template <bool FTZ>
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  if (FTZ)
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  else
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Of a value that is 0 or normal, as its reciprocal is.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <typename PT, typename GT, bool kSmall, int TENSORS>
__global__ void __launch_bounds__(kThreads<kSmall>) adamw_kernel(const __grid_constant__ AdamTable<TENSORS> a) {
  pdl_launch_dependents();
  pdl_wait();
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= (int)blockIdx.x) lo = mid; else hi = mid;
  }
  const AdamEntry &t = a.t[lo];
  const int64_t n = t.n, base = (int64_t)((int)blockIdx.x - a.first[lo]) * kChunk<kSmall>;
  const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.0f;
  // a round's loads are issued before the round before is worked on (352 M
  // values with 8-bit states: 871 us instead of 1104; four rounds 1038, fewer
  // registers for more blocks 1003 or worse; with a reciprocal for the
  // quotient, flushing roots, and the tests on values joined over a thread's 8: 843)
  struct Loaded {
    Raw8<PT> p;
    Raw8<GT> g;
    Raw8<float> m, v;           // float32 states
    uint2 mc, vc;               // 8-bit states
    uint32_t ms, vs;
  };
  auto load = [&](int64_t i) {
    Loaded x;
    const int live = (int)(n - i < 0 ? 0 : n - i < 8 ? n - i : 8);
    if (live > 0) {
      x.p = load_raw(static_cast<const PT *>(t.p) + i, live);
      x.g = load_raw(static_cast<const GT *>(t.g) + i, live);
      if (kSmall) {
        x.mc = load_codes(static_cast<const uint8_t *>(t.m) + i, live);
        x.vc = load_codes(static_cast<const uint8_t *>(t.v) + i, live);
        x.ms = t.ms[i >> 5];
        x.vs = t.vs[i >> 5];
      } else {
        x.m = load_raw(static_cast<const float *>(t.m) + i, live);
        x.v = load_raw(static_cast<const float *>(t.v) + i, live);
      }
    }
    return x;
  };
  int64_t i = base + (int64_t)threadIdx.x * 8;
  Loaded ahead = load(i);
#pragma unroll
  for (int r = 0; r < kRounds; ++r, i += 8 * kThreads<kSmall>) {
    if (kSmall ? i - 8 * (threadIdx.x & 31) >= n : i >= n) break;      // 8-bit states: whole warps go on
    const int live = (int)(n - i < 0 ? 0 : n - i < 8 ? n - i : 8);
    const Loaded x = ahead;
    if (r + 1 < kRounds) ahead = load(i + 8 * kThreads<kSmall>);
    V8 p, g, m, v, root;
    // the least v above zero, as its bits less one (0: the largest of all)
    uint32_t low = 0xffffffffu;
    constexpr uint32_t kLeastNormal = 0x00800000u - 1u;
    if (!kSmall || live > 0) {
      p = x.p.get();
      g = x.g.get();
      m = kSmall ? decode8(x.mc, x.ms) : x.m.get();
      v = kSmall ? decode8(x.vc, x.vs) : x.v.get();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // each product and sum of m and v rounded by itself (no fused
        // multiply-add), so that the 8-bit codes have one right answer
        const float gj = __fmul_rn(g.v[j], gs);
        const float old = kSmall ? __fmul_rn(v.v[j], v.v[j]) : v.v[j];
        m.v[j] = __fadd_rn(__fmul_rn(m.v[j], a.beta1), __fmul_rn(gj, a.one_minus_beta1));
        v.v[j] = __fadd_rn(__fmul_rn(old, a.beta2), __fmul_rn(__fmul_rn(gj, gj), a.one_minus_beta2));
        root.v[j] = sqrt_approx<kSmall>(v.v[j]);
        low = min(low, __float_as_uint(v.v[j]) - 1u);
      }
      if (kSmall && low < kLeastNormal) {
#pragma unroll
        for (int j = 0; j < 8; ++j) root.v[j] = __fsqrt_rn(v.v[j]);
      }
      // a root is 0 or at least 2^-75, so the sum is 0 or normal.  An approximate
      // root (float32 states too), an approximate reciprocal and the products leave
      // the update within 2^-21 of itself: less than p's own rounding unless p is
      // smaller than eight updates
#pragma unroll
      for (int j = 0; j < 8; ++j)
        p.v[j] = p.v[j] * a.keep - a.rate * (m.v[j] * rcp_approx(fmaf(root.v[j], a.root_scale, a.eps)));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) p.v[j] = m.v[j] = v.v[j] = root.v[j] = 0.f;
    }
    if (kSmall) {
      // scales: the root of the largest v is the largest root
      float m_max = 0.f, v_max = 0.f;
      // a code that is not subnormal changes where a root passes an odd multiple
      // of 2^19 units of its last place; the approximate root decides unless it is
      // that near (about one value in 200 000; even multiples are the codes
      // themselves, which a BF16 gradient that equals the held root hits often)
      uint32_t near = 0xffffffffu;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m_max = fmaxf(m_max, fabsf(m.v[j]));
        v_max = fmaxf(v_max, v.v[j]);
        near = min(near, (__float_as_uint(root.v[j]) + 2u + (1u << 19)) << 12);
      }
      const int me = ue8m0_exponent<true>(group_max(m_max)), ve = ue8m0_exponent<true>(__fsqrt_rn(group_max(v_max)));
      const uint8_t mb = (uint8_t)(me + 127), vb = (uint8_t)(ve + 127);
      // subnormal codes are below 2^-6 of the scale; a root above zero takes at
      // least the smallest, 2^-9
      const float unit = scale_of(vb), subnormal = unit * 0.015625f, least = unit * 0.001953125f;
      if (near < (5u << 12) || low < max(__float_as_uint(1.01f * subnormal * subnormal), kLeastNormal)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          root.v[j] = __fsqrt_rn(v.v[j]);
          if (root.v[j] > 0.f) root.v[j] = fmaxf(root.v[j], least);
        }
      }
      const uint2 mc = encode8(m, me), vc = encode8(root, ve);
      if (live > 0) {
        store_codes(static_cast<uint8_t *>(t.m) + i, mc, live);
        store_codes(static_cast<uint8_t *>(t.v) + i, vc, live);
        if ((i & 31) == 0) {
          t.ms[i >> 5] = mb;
          t.vs[i >> 5] = vb;
        }
      }
    } else {
      store_some(static_cast<float *>(t.m) + i, m, live);
      store_some(static_cast<float *>(t.v) + i, v, live);
    }
    if (!kSmall || live > 0) {
      store_some(static_cast<PT *>(t.p) + i, p, live);
      if (t.copy) store_some(t.copy + i, p, live);
    }
  }
}

template <typename PT, typename GT, bool kSmall, int TENSORS>
int launch_some(const moe_adamw_args &a, int from, int to, cudaStream_t st) {
  AdamTable<TENSORS> t;
  t.count = 0;
  int64_t blocks = 0;
  for (int i = from; i < to; ++i) {
    const moe_adamw_tensor &x = a.tensors[i];
    if (x.n == 0) continue;
    t.t[t.count] = AdamEntry{x.n, x.p, x.g, x.m, x.v, x.m_scale, x.v_scale, x.copy};
    t.first[t.count++] = (int)blocks;
    blocks += ceil_div(x.n, kChunk<kSmall>);
  }
  if (blocks == 0) return MOE_OK;
  t.first[t.count] = (int)blocks;
  t.beta1 = (float)a.beta1;
  t.one_minus_beta1 = (float)(1.0 - a.beta1);
  t.beta2 = (float)a.beta2;
  t.one_minus_beta2 = (float)(1.0 - a.beta2);
  t.keep = (float)(1.0 - a.lr * a.weight_decay);
  t.rate = (float)(a.lr / (1.0 - std::pow(a.beta1, (double)a.step)));
  t.root_scale = (float)(1.0 / std::sqrt(1.0 - std::pow(a.beta2, (double)a.step)));
  t.eps = a.eps > 0 ? std::max((float)a.eps, 1.17549435e-38f) : 0.f;       // 0 or normal (rcp_approx)
  t.grad_scale = a.grad_scale;
  return launch_pdl(adamw_kernel<PT, GT, kSmall, TENSORS>, dim3((unsigned)blocks), dim3(kThreads<kSmall>), 0, st, t);
}

constexpr int kFew = 40, kMany = 400;       // tensors per launch: 3 KB or 28 KB of kernel parameters
static_assert(sizeof(AdamTable<kFew>) <= 4000 && sizeof(AdamTable<kMany>) <= 32000, "kernel parameter space");

// Launches of at most kMany tensors and less than 2^31 blocks each.
template <typename PT, typename GT, bool kSmall>
int step_all(const moe_adamw_args &a, cudaStream_t st) {
  for (int from = 0; from < a.n_tensors;) {
    int to = from;
    int64_t blocks = 0;
    while (to < a.n_tensors && to - from < kMany) {
      const int64_t more = ceil_div(a.tensors[to].n, kChunk<kSmall>);
      if (to > from && blocks + more > 0x7fffffffLL) break;
      blocks += more;
      ++to;
    }
    const int rc = to - from <= kFew ? launch_some<PT, GT, kSmall, kFew>(a, from, to, st)
                                     : launch_some<PT, GT, kSmall, kMany>(a, from, to, st);
    if (rc != MOE_OK) return rc;
    from = to;
  }
  return MOE_OK;
}

template <typename PT, typename GT>
int step_bits(const moe_adamw_args &a, cudaStream_t st) {
  return a.state_bits == 8 ? step_all<PT, GT, true>(a, st) : step_all<PT, GT, false>(a, st);
}

template <typename PT>
int step_grad(const moe_adamw_args &a, cudaStream_t st) {
  return a.g_dtype == MOE_F32 ? step_bits<PT, float>(a, st) : step_bits<PT, uint16_t>(a, st);
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" int moe_adamw_step(const moe_adamw_args *a, cudaStream_t stream) {
  if (!a || a->struct_size != sizeof(moe_adamw_args) || a->n_tensors < 0) return MOE_ERR_INVALID_ARG;
  if ((a->p_dtype != MOE_BF16 && a->p_dtype != MOE_F32) || (a->g_dtype != MOE_BF16 && a->g_dtype != MOE_F32))
    return MOE_ERR_INVALID_ARG;
  if ((a->state_bits != 32 && a->state_bits != 8) || a->step < 1) return MOE_ERR_INVALID_ARG;
  if (!(a->beta1 >= 0 && a->beta1 < 1 && a->beta2 >= 0 && a->beta2 < 1 && a->eps >= 0) || !std::isfinite(a->eps) ||
      !std::isfinite(a->lr) || !std::isfinite(a->weight_decay))
    return MOE_ERR_INVALID_ARG;
  if (a->n_tensors == 0) return MOE_OK;
  if (!a->tensors) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->grad_scale, 4)) return MOE_ERR_MISALIGNED;
  for (int i = 0; i < a->n_tensors; ++i) {
    const moe_adamw_tensor &t = a->tensors[i];
    if (t.n < 0) return MOE_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (ceil_div(t.n, a->state_bits == 8 ? kChunk<true> : kChunk<false>) > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!t.p || !t.g || !t.m || !t.v || (a->state_bits == 8 && (!t.m_scale || !t.v_scale)) ||
        (t.copy && a->p_dtype == MOE_BF16))
      return MOE_ERR_INVALID_ARG;
    if (!aligned(t.p, 16) || !aligned(t.g, 16) || !aligned(t.m, 16) || !aligned(t.v, 16) || !aligned(t.copy, 16))
      return MOE_ERR_MISALIGNED;
  }
  return a->p_dtype == MOE_F32 ? step_grad<float>(*a, stream) : step_grad<uint16_t>(*a, stream);
}
