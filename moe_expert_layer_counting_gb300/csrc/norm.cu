// norm.cu -- the norms before and after the expert layer with its gate and
// residual scale, and their gradients (include/moe_norm.h has the formulas).
//
// Both directions are bound by HBM if the SM keeps up: every row is read once
// and written once, but a row needs two sums over its columns one after the
// other, and ~17 operations a value in the backward pass.  So:
//   - a group of H / 16 threads owns a row at a time, a thread 16 columns (with 8,
//     the instructions that do not depend on the columns are as many as those
//     that do: 149 instead of 127 us for the gradients of 8192 x 7168 in BF16);
//   - the rows to come are copied (bulk copies) into a ring in shared memory; a
//     row is taken into registers, and its slot has its next row on the way
//     before the row's first sum is used;
//   - arithmetic on pairs (f32x2 instructions), and column constants (the
//     weights with their offset, the channel gate) made once per block;
//   - the gradients of w_post and of a channel gate are the same column sum
//     sum_t d b rsqrt(mean b^2 + eps), times a constant of the column.
// A row of more than 8192 columns is split over the two blocks of a cluster
// (SPLIT), which add their sums through each other's shared memory (2048 x 16384:
// 53 and 84 us; held in one block's registers it took 69 and 214).  One row of
// those is in work per cluster, and each of its two sums crosses to the other
// block and is waited for, which the floors (40 and 59 us) have none of.
// Measured, BF16, channel gate: forward of 8192 x 7168 in 74 us (6.3 TB/s), the
// gradients in 125 us (5.6 TB/s); 4096 x 7168 in 41 and 70 us, of which ~10 us
// are the first rows' way in, the last ones' way out and the sums of the parts.
#include <cuda_bf16.h>

#include <atomic>
#include <cstdlib>

#include "../../include/moe_norm.h"
#include "host_common.h"
#include "pairs.cuh"
#include "ptx.cuh"
#include "row_sums.cuh"

namespace mxq {

namespace {

constexpr int kMaxH = 16384;

struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 unpack_bf16x8(const uint4 &q) {
  F8 f;
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[2 * i] = bf16_bits_to_float(w[i] & 0xFFFFu);
    f.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return f;
}

// Eight values of a row as they lie in memory (registers until they are used).
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> {
  uint4 q;
  __device__ __forceinline__ void load(const uint16_t *p) { q = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ P2 two(int i) const { return from_bf16x2(i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w); }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ F8 get() const { return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
  __device__ __forceinline__ P2 two(int i) const {
    return i == 0 ? pair(a.x, a.y) : i == 1 ? pair(a.z, a.w) : i == 2 ? pair(b.x, b.y) : pair(b.z, b.w);
  }
};

__device__ __forceinline__ void store_pairs(uint16_t *p, const P2 (&v)[4]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(to_bf16x2(v[0]), to_bf16x2(v[1]), to_bf16x2(v[2]), to_bf16x2(v[3]));
}
__device__ __forceinline__ void store_pairs(float *p, const P2 (&v)[4]) {
  const float2 a = split(v[0]), b = split(v[1]), c = split(v[2]), d = split(v[3]);
  reinterpret_cast<float4 *>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
  reinterpret_cast<float4 *>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
}

// Eight values of a weight or gate, of either type (the same branch for the
// whole launch).
__device__ __forceinline__ F8 load8_any(const void *p, int dtype, int64_t i) {
  if (dtype == MOE_BF16) return unpack_bf16x8(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i)));
  const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
  const float4 a = __ldg(q), b = __ldg(q + 1);
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ float load1_any(const void *p, int dtype, int64_t i) {
  return dtype == MOE_BF16 ? bf16_bits_to_float(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store1_any(void *p, int dtype, int64_t i, float v) {
  if (dtype == MOE_BF16)
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float *>(p)[i] = v;
}

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// ---------------------------------------------------------------- rows through a ring in shared memory

// A launch: `group` threads a row (a multiple of 32), `groups` rows at a time
// in a block, `stages` slots a group; `inject_wait`: the debug hook's wait.
struct RingShape {
  int group, groups, stages, inject_wait;
};
constexpr int kThreads = 512;                           // of a block, at most
constexpr int V = 2;                                    // 8-column vectors of a thread
constexpr int kMaxGroups = 4, kMaxStages = 8;
constexpr long long kRingLimit = 2000000000LL;          // ~1 s
constexpr long long kInjectedLimit = 20000000LL;        // ~10 ms: the debug hook's

// One row tensor of a launch: where its row t is, its bytes, its place in a slot.
struct RowSource {
  const char *base;
  int64_t stride;              // bytes
  int bytes;                   // of a row; 0: not read
  int at;
};

struct RingSmem {
  uint64_t full[kMaxGroups][kMaxStages];
  float red[kMaxGroups][2][2][4 * 32];                  // of even and odd rows, two sums each
  float4 other[2][2];                                   // SPLIT: the other block's, the same four
  uint64_t here[2][2];                                  //        and the arrival of each
};

template <int N>
__device__ __forceinline__ int place_rows(RowSource (&src)[N]) {
  int at = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    src[i].at = at;
    at += src[i].bytes;
  }
  return at;
}

template <bool SPLIT, int N>
__device__ __forceinline__ void ring_init(RingSmem &sm, const RingShape &sh, const RowSource (&src)[N]) {
  for (int i = (int)threadIdx.x; i < kMaxGroups * 2 * 2 * 4 * 32; i += (int)blockDim.x) (&sm.red[0][0][0][0])[i] = 0.f;
  if (threadIdx.x == 0) {
    uint32_t copies = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) copies += src[i].bytes > 0 ? 1u : 0u;
    for (int g = 0; g < sh.groups; ++g)
      for (int s = 0; s < sh.stages; ++s) mbar_init(&sm.full[g][s], copies);
    if (SPLIT)
      for (int i = 0; i < 4; ++i) mbar_init(&sm.here[i >> 1][i & 1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (SPLIT) cluster_sync();
}

// Which tensors' copies this thread issues: each by the first lane of a warp of
// its own (a thread's copies issue one after another), as far as the group has
// warps.
template <int N>
__device__ __forceinline__ uint32_t my_copies(const RowSource (&src)[N], int warps, int warp) {
  uint32_t mask = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (src[i].bytes > 0 && i % warps == warp && (threadIdx.x & 31) == 0) mask |= 1u << i;
  return mask;
}

// 16 bytes into another block's shared memory, counted by its barrier.
__device__ __forceinline__ void send16(uint32_t to, uint32_t bar, const float4 &f) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
               "f"(f.x), "f"(f.y), "f"(f.z), "f"(f.w), "r"(bar)
               : "memory");
}

// Row t into a slot.
template <int N>
__device__ __forceinline__ void ring_copy(uint32_t mask, const RowSource (&src)[N], unsigned char *slot, uint64_t *bar,
                                          int64_t t) {
  if (mask == 0) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!(mask >> i & 1u)) continue;
    mbar_arrive_expect_tx(bar, (uint32_t)src[i].bytes);
    bulk_load(slot + src[i].at, src[i].base + t * src[i].stride, (uint32_t)src[i].bytes, bar);
  }
}

// Waits for this block's own copies (or the other's sums).  After one that gives
// up, and is reported where the call has status words, the thread begins no other
// and no more copies (it has none `ahead`), and gives those in flight time to land
// before it leaves.  All but the first look is out of line: inside the loop it
// changes how the rest is scheduled (gradients of 2048 x 16384: 84 us, or 96).
constexpr unsigned kGaveUp = ~0u;

__device__ __noinline__ bool ring_wait_longer(uint64_t *bar, uint32_t parity, int *status) {
  const long long t0 = clock64();
  bool last;
  do {
    last = clock64() - t0 >= kRingLimit;
    if (mbar_try_wait(bar, parity)) return true;
  } while (!last);
  report_status(status, kStatusTimeout);
  return false;
}
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity, int *status) {
  return mbar_try_wait(bar, parity) || ring_wait_longer(bar, parity, status);
}
// The debug hook: the launch's first thread begins with a wait that runs out.
__device__ __noinline__ bool injected_wait(int *status) {
  if (blockIdx.x != 0 || threadIdx.x != 0) return false;
  const long long t0 = clock64();
  while (clock64() - t0 < kInjectedLimit) __nanosleep(1000);
  report_status(status, kStatusTimeout);
  return true;
}
__device__ __forceinline__ void let_land() {
  const long long t0 = clock64();
  while (clock64() - t0 < 200000) __nanosleep(1000);      // ~100 us
}

// Sums over a split row, from the sums over this block's columns: the first
// thread of each block writes its own into the other's shared memory, and both
// add the two in the order of the columns.  A place is written again two rows
// later, after this block's sums of the row between, that is after all its
// threads have read it.
template <int N>
__device__ __forceinline__ bool add_other(float (&v)[N], RingSmem &sm, int turn, int which, uint32_t parity, uint32_t rank,
                                          int *status) {
  uint64_t *bar = &sm.here[turn][which];
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(bar, 16);
    send16(mapa_shared(smem_u32(&sm.other[turn][which]), rank ^ 1), mapa_shared(smem_u32(bar), rank ^ 1),
           make_float4(v[0], v[1 % N], v[2 % N], 0.f));
  }
  if (!ring_wait(bar, parity, status)) {
    v[0] = __int_as_float(0x7fffffff);
    return false;
  }
  const float4 o = sm.other[turn][which];
  const float f[3] = {o.x, o.y, o.z};
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = rank == 0 ? v[k] + f[k] : f[k] + v[k];
  return true;
}

// Column constants in shared memory: 8 columns of vector c in two planes, so
// that neighbouring threads' 16-byte reads do not share banks.
__device__ __forceinline__ void put_columns(float4 *plane, int vecs, int c, const F8 &f) {
  plane[c] = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  plane[vecs + c] = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}
__device__ __forceinline__ void get_columns(const float4 *plane, int vecs, int c, P2 (&w)[4]) {
  const float4 a = plane[c], b = plane[vecs + c];
  w[0] = pair(a.x, a.y);
  w[1] = pair(a.z, a.w);
  w[2] = pair(b.x, b.y);
  w[3] = pair(b.z, b.w);
}

// weight_offset + w, or 1 without a weight.
__device__ __forceinline__ F8 offset_weight(const void *w, int dtype, int c, float offset) {
  F8 f;
  if (w) {
    f = load8_any(w, dtype, 8 * c);
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] += offset;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = 1.0f;
  }
  return f;
}
__device__ __forceinline__ F8 gate8(const void *gate, int dtype, bool sig, int64_t i) {
  F8 f = load8_any(gate, dtype, i);
  if (sig)
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = sigmoid(f.v[j]);
  return f;
}
// A full gate's 8 values from the ring.
__device__ __forceinline__ F8 ring_gate8(const unsigned char *row, int c, int dtype, bool sig) {
  F8 f;
  if (dtype == MOE_BF16) {
    f = unpack_bf16x8(*reinterpret_cast<const uint4 *>(row + 16 * c));
  } else {
    Raw8<float> r;
    r.load(reinterpret_cast<const float *>(row) + 8 * c);
    f = r.get();
  }
  if (sig)
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = sigmoid(f.v[j]);
  return f;
}
__device__ __forceinline__ void to_pairs(const F8 &f, P2 (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pair(f.v[2 * i], f.v[2 * i + 1]);
}
__device__ __forceinline__ float total(P2 p) {
  const float2 f = split(p);
  return f.x + f.y;
}

// FULL: a gate of each value.  ALL: a layer's answer, both norms and both outputs
// are there (the branches on them cost as much as the arithmetic).
template <typename XT, bool FULL, bool ALL, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    norm_forward_kernel(const __grid_constant__ moe_norm_args a, const RingShape sh) {
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ RingSmem sm;
  // this block's columns: 8 vecs of them, from 8 c0 on; the rows go by clusters
  const int H = (int)a.H, half = (H + 8) >> 4;
  const uint32_t rank = SPLIT ? cluster_ctarank() : 0;
  const int c0 = rank * half, vecs = SPLIT ? (rank == 0 ? half : (H >> 3) - half) : H >> 3, cols = SPLIT ? 8 * vecs : H;
  const unsigned block = SPLIT ? blockIdx.x >> 1 : blockIdx.x, blocks = SPLIT ? gridDim.x >> 1 : gridDim.x;
  const bool sig = a.gate_sigmoid != 0;
  const bool has_b = ALL || a.b, post = ALL || a.w_post, out_y = ALL || (a.b && a.y), out_n = ALL || a.n;
  const int gate_size = a.gate_dtype == MOE_F32 ? 4 : 2;
  const int xb = cols * (int)sizeof(XT);
  RowSource src[3] = {
      {static_cast<const char *>(a.x) + 8 * c0 * (int)sizeof(XT), a.ldx * (int64_t)sizeof(XT), xb, 0},
      {reinterpret_cast<const char *>(a.b) + 16 * c0, a.ldb * 2, has_b ? cols * 2 : 0, 0},
      {static_cast<const char *>(a.gate) + 8 * c0 * gate_size, a.ld_gate * gate_size, FULL ? cols * gate_size : 0, 0}};
  const int row_bytes = place_rows(src);
  const int group = (int)threadIdx.x / sh.group, tid = (int)threadIdx.x - group * sh.group;
  const int warps = sh.group >> 5, warp = tid >> 5;
  const unsigned T = (unsigned)a.T, first = block * (unsigned)sh.groups + (unsigned)group,
                 n = blocks * (unsigned)sh.groups;
  unsigned ahead = (unsigned)sh.stages * n;
  unsigned char *ring = ring_smem + (size_t)group * sh.stages * row_bytes;
  const uint32_t copies = my_copies(src, warps, warp);
  ring_init<SPLIT>(sm, sh, src);
  pdl_launch_dependents();
  pdl_wait();
  for (int s = 0; s < sh.stages; ++s)
    if (first + s * n < T) ring_copy(copies, src, ring + s * row_bytes, &sm.full[group][s], first + s * n);
  if (a.status && blockIdx.x == 0 && threadIdx.x < 16) a.status[threadIdx.x] = 0;
  const float inv_h = 1.0f / (float)H;
  auto sync = [&] {                        // converged warps, or after shuffles
    if (warps == 1) __syncwarp(); else named_bar_sync(1 + group, sh.group);
  };
  // the weight after the layer times a channel gate; the weight before the next
  P2 c_post[V][4], c_pre[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * sh.group;
    if (c >= vecs) continue;
    F8 f = offset_weight(a.w_post, a.w_dtype, c0 + c, a.weight_offset);
    if (a.gate_kind == MOE_GATE_CHANNEL) {
      const F8 z = gate8(a.gate, a.gate_dtype, sig, 8 * (c0 + c));
#pragma unroll
      for (int j = 0; j < 8; ++j) f.v[j] *= z.v[j];
    }
    to_pairs(f, c_post[i]);
    to_pairs(offset_weight(a.w_pre, a.w_dtype, c0 + c, a.weight_offset), c_pre[i]);
  }
  P2 scale = twice(a.b ? a.residual_scale : 1.0f);
  // After a wait gave up the thread's terms are NaN, in its columns and in its
  // rows' sums: no output is wrong and looks right.
  float zero = 0.f;
  auto give_up = [&] {
    ahead = kGaveUp;
    zero = __int_as_float(0x7fffffff);
    scale = twice(zero);
  };
  XT *py = static_cast<XT *>(a.y) + first * a.ldy + 8 * (c0 + tid);
  uint16_t *pn = a.n + first * a.ldn + 8 * (c0 + tid);
  const int64_t step_y = n * a.ldy, step_n = n * a.ldn;
  if (sh.inject_wait && injected_wait(a.status)) give_up();
  __syncwarp();
  int stage = 0, turn = 0;
  uint32_t phase = 0, half_phase = 0;      // half_phase: of this turn's sums of a split row
  for (unsigned t = first; t < T; t += n, half_phase ^= (uint32_t)turn, turn ^= 1) {
    unsigned char *row = ring + stage * row_bytes;
    if (ahead != kGaveUp && !ring_wait(&sm.full[group][stage], phase, a.status)) give_up();
    P2 y[V][4], u[V][4], sq = twice(zero);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * sh.group;
      if (c >= vecs) continue;
      Raw8<XT> x;
      x.load(reinterpret_cast<const XT *>(row) + 8 * c);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[i][k] = scale * x.two(k);
      if (has_b) {
        Raw8<uint16_t> b;
        b.load(reinterpret_cast<const uint16_t *>(row + src[1].at) + 8 * c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u[i][k] = b.two(k);
          sq = fma2(u[i][k], u[i][k], sq);
          u[i][k] = u[i][k] * c_post[i][k];
        }
        if (FULL) {
          P2 z[4];
          to_pairs(ring_gate8(row + src[2].at, c, a.gate_dtype, sig), z);
#pragma unroll
          for (int k = 0; k < 4; ++k) u[i][k] = u[i][k] * z[k];
        }
      }
    }
    float rb = 1.0f;
    if (post) {
      float s[1] = {total(sq)};
      group_sum(s, warps, warp, sm.red[group][turn][0], sync);
      if (SPLIT && ahead != kGaveUp && !add_other(s, sm, turn, 0, half_phase, rank, a.status)) give_up();
      rb = rsqrtf(s[0] * inv_h + a.eps);
    } else {
      __syncwarp();
      sync();
    }
    // the row is in registers: its slot takes the row after the ring's
    if (T - t > ahead) ring_copy(copies, src, row, &sm.full[group][stage], t + ahead);
    if (++stage == sh.stages) { stage = 0; phase ^= 1; }
    if (a.gate_kind == MOE_GATE_TOKEN) {
      const float z = load1_any(a.gate, a.gate_dtype, t);
      rb *= sig ? sigmoid(z) : z;
    }
    sq = twice(zero);
    const P2 rb2 = twice(rb);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (tid + i * sh.group >= vecs) continue;
      if (has_b) {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[i][k] = fma2(u[i][k], rb2, y[i][k]);
        if (out_y) store_pairs(py + 8 * i * sh.group, y[i]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) sq = fma2(y[i][k], y[i][k], sq);
    }
    py += step_y;
    if (!out_n) continue;
    float s[1] = {total(sq)};
    group_sum(s, warps, warp, sm.red[group][turn][1], sync);
    if (SPLIT && ahead != kGaveUp && !add_other(s, sm, turn, 1, half_phase, rank, a.status)) give_up();
    const P2 r2 = twice(rsqrtf(s[0] * inv_h + a.eps));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (tid + i * sh.group >= vecs) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) y[i][k] = y[i][k] * r2 * c_pre[i][k];
      store_pairs(pn + 8 * i * sh.group, y[i]);
    }
    pn += step_n;
  }
  if (ahead == kGaveUp) let_land();
  if (SPLIT) {                             // the other block may still write into this one's memory
    __syncthreads();
    cluster_sync();
  }
}

// Column sums over rows: of dn h (dw_pre) and of S = d b rsqrt(mean b^2 + eps)
// (times a token's or a value's gate), from which norm_parts_kernel makes
// dw_post and a channel gate's dgate.  Each thread adds up its group's rows in
// registers, in row order, a block adds its groups' sums in order and leaves one
// part; norm_parts_kernel adds the parts in block order.
enum : int { kSumPre = 0, kSumPost = 1 };

// FULL, ALL as above (ALL: and all gradients of rows).  Values stay in
// registers as they lie in memory: a spilled register goes through the little
// L1 that the ring leaves, and costs more than unpacking twice (the form with a
// float32 stream and a full gate spills 80 bytes all the same: 160 us at 4096 x
// 7168, floor 95).  A float32 dy is
// loaded directly, from L2 where its row was brought one row before: with it in
// the ring, a slot of 7168 columns fits only once.  With a full gate or a
// float32 stream the row is read again from its slot after the first sum
// (kLate), and the slot is free after the second.
template <typename XT, bool FULL, bool ALL, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    norm_backward_kernel(const __grid_constant__ moe_norm_args a, const __grid_constant__ moe_norm_grads g,
                         const RingShape sh, int *status, float *parts) {
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ RingSmem sm;
  // this block's columns: 8 vecs of them, from 8 c0 on; the rows go by clusters
  const int H = (int)a.H, half = (H + 8) >> 4;
  const uint32_t rank = SPLIT ? cluster_ctarank() : 0;
  const int c0 = rank * half, vecs = SPLIT ? (rank == 0 ? half : (H >> 3) - half) : H >> 3, cols = SPLIT ? 8 * vecs : H;
  const unsigned block = SPLIT ? blockIdx.x >> 1 : blockIdx.x, blocks = SPLIT ? gridDim.x >> 1 : gridDim.x;
  const bool token = a.gate_kind == MOE_GATE_TOKEN, sig = a.gate_sigmoid != 0;
  const bool has_b = ALL || a.b, post = ALL || a.w_post, pre = ALL || a.w_pre, has_dy = ALL || g.dy, out_dx = ALL || g.dx,
             out_db = ALL || g.db;
  constexpr bool kDirect = sizeof(XT) == 4, kLate = FULL || kDirect;
  const int xb = cols * (int)sizeof(XT), gate_size = a.gate_dtype == MOE_F32 ? 4 : 2;
  RowSource src[5] = {
      {static_cast<const char *>(a.x) + 8 * c0 * (int)sizeof(XT), a.ldx * (int64_t)sizeof(XT), pre ? xb : 0, 0},
      {reinterpret_cast<const char *>(g.dn) + 16 * c0, g.ld_dn * 2, pre ? cols * 2 : 0, 0},
      {static_cast<const char *>(g.dy) + 8 * c0 * (int)sizeof(XT), g.ld_dy * (int64_t)sizeof(XT),
       has_dy && !kDirect ? xb : 0, 0},
      {reinterpret_cast<const char *>(a.b) + 16 * c0, a.ldb * 2, has_b ? cols * 2 : 0, 0},
      {static_cast<const char *>(a.gate) + 8 * c0 * gate_size, a.ld_gate * gate_size, FULL ? cols * gate_size : 0, 0}};
  const int row_bytes = place_rows(src);
  const int group = (int)threadIdx.x / sh.group, tid = (int)threadIdx.x - group * sh.group;
  const int warps = sh.group >> 5, warp = tid >> 5;
  const unsigned T = (unsigned)a.T, first = block * (unsigned)sh.groups + (unsigned)group,
                 n = blocks * (unsigned)sh.groups;
  unsigned ahead = (unsigned)sh.stages * n;
  // column constants, then the rings
  float4 *c_pre = reinterpret_cast<float4 *>(ring_smem), *c_post = c_pre + 2 * vecs;
  unsigned char *ring = ring_smem + 2 * cols * 4 + (size_t)group * sh.stages * row_bytes;
  const uint32_t copies = my_copies(src, warps, warp);
  ring_init<SPLIT>(sm, sh, src);
  pdl_launch_dependents();
  pdl_wait();
  for (int s = 0; s < sh.stages; ++s)
    if (first + s * n < T) ring_copy(copies, src, ring + s * row_bytes, &sm.full[group][s], first + s * n);
  if (blockIdx.x == 0 && threadIdx.x < 16) status[threadIdx.x] = 0;
  for (int c = (int)threadIdx.x; c < vecs; c += (int)blockDim.x) {
    put_columns(c_pre, vecs, c, offset_weight(a.w_pre, a.w_dtype, c0 + c, a.weight_offset));
    F8 f = offset_weight(a.w_post, a.w_dtype, c0 + c, a.weight_offset);
    if (a.gate_kind == MOE_GATE_CHANNEL) {
      const F8 z = gate8(a.gate, a.gate_dtype, sig, 8 * (c0 + c));
#pragma unroll
      for (int j = 0; j < 8; ++j) f.v[j] *= z.v[j];
    }
    put_columns(c_post, vecs, c, f);
  }
  __syncthreads();
  const float inv_h = 1.0f / (float)H;
  auto sync = [&] {                        // converged warps, or after shuffles
    if (warps == 1) __syncwarp(); else named_bar_sync(1 + group, sh.group);
  };
  P2 sum_pre[V][4], sum_post[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) sum_pre[i][k] = sum_post[i][k] = twice(0.f);
  const P2 scale = twice(a.b ? a.residual_scale : 1.0f);
  XT *px = static_cast<XT *>(g.dx) + first * g.ld_dx + 8 * (c0 + tid);
  uint16_t *pb = g.db + first * g.ld_db + 8 * (c0 + tid);
  const int64_t step_x = n * g.ld_dx, step_b = n * g.ld_db;
  const XT *pd = static_cast<const XT *>(g.dy) + first * g.ld_dy + 8 * (c0 + tid);
  const int64_t step_d = n * g.ld_dy;
  if (sh.inject_wait && injected_wait(status)) ahead = kGaveUp;
  __syncwarp();
  int stage = 0, turn = 0;
  uint32_t phase = 0, half_phase = 0;      // half_phase: of this turn's sums of a split row
  for (unsigned t = first; t < T; t += n, half_phase ^= (uint32_t)turn, turn ^= 1) {
    unsigned char *row = ring + stage * row_bytes;
    uint64_t *full = &sm.full[group][stage];
    Raw8<XT> y[V], dy[V];
    Raw8<uint16_t> dn[V], b[V];
    if (kDirect && has_dy) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (tid + i * sh.group < vecs) dy[i].load(pd + 8 * i * sh.group);
      pd += step_d;
      if (tid == 0 && T - t > n) prefetch_l2_bulk(pd, (uint32_t)xb);
    }
    if (ahead != kGaveUp && !ring_wait(full, phase, status)) ahead = kGaveUp;
    // sums of y^2, dn w y and b^2
    P2 s0 = twice(0.f), s1 = s0, s2 = s0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * sh.group;
      if (c >= vecs) continue;
      if (pre) {
        y[i].load(reinterpret_cast<const XT *>(row) + 8 * c);
        dn[i].load(reinterpret_cast<const uint16_t *>(row + src[1].at) + 8 * c);
        P2 w[4];
        get_columns(c_pre, vecs, c, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s0 = fma2(y[i].two(k), y[i].two(k), s0);
          s1 = fma2(dn[i].two(k) * w[k], y[i].two(k), s1);
        }
      }
      if (!kDirect && has_dy) dy[i].load(reinterpret_cast<const XT *>(row + src[2].at) + 8 * c);
      if (has_b) {
        b[i].load(reinterpret_cast<const uint16_t *>(row + src[3].at) + 8 * c);
#pragma unroll
        for (int k = 0; k < 4; ++k) s2 = fma2(b[i].two(k), b[i].two(k), s2);
      }
    }
    float s[3] = {total(s0), total(s1), total(s2)};
    group_sum(s, warps, warp, sm.red[group][turn][0], sync);
    if (SPLIT && ahead != kGaveUp && !add_other(s, sm, turn, 0, half_phase, rank, status)) ahead = kGaveUp;
    // the row is in registers: its slot takes the row after the ring's
    if (!kLate && T - t > ahead) ring_copy(copies, src, row, full, t + ahead);
    if (++stage == sh.stages) { stage = 0; phase ^= 1; }
    const float r = rsqrtf(s[0] * inv_h + a.eps);
    const float rb = post ? rsqrtf(s[2] * inv_h + a.eps) : 1.0f;
    float gate_t = 1.0f;
    if (token) {
      gate_t = load1_any(a.gate, a.gate_dtype, t);
      if (sig) gate_t = sigmoid(gate_t);
    }
    const P2 rs = twice(rb * gate_t);
    // r times mean(dn w h); the row's magnitude cancels factor by factor (r cubed
    // would leave the range of float32 for rows below 1e-13 or above 1e13)
    const P2 r2 = twice(r), back = twice(-r * (r * s[1] * inv_h));
    P2 d[V][4], q2 = twice(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * sh.group;
      if (c >= vecs) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) d[i][k] = has_dy ? dy[i].two(k) : twice(0.f);
      if (pre) {
        // d += r (dn w - h mean(dn w h)), h = y r
        if (kLate) {
          y[i].load(reinterpret_cast<const XT *>(row) + 8 * c);
          dn[i].load(reinterpret_cast<const uint16_t *>(row + src[1].at) + 8 * c);
        }
        P2 w[4];
        get_columns(c_pre, vecs, c, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const P2 g = dn[i].two(k), f = y[i].two(k);
          d[i][k] = fma2(fma2(f, back, g * w[k]), r2, d[i][k]);
          sum_pre[i][k] = fma2(g * r2, f, sum_pre[i][k]);
        }
      }
      if (out_dx) {
        P2 o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = d[i][k] * scale;
        store_pairs(px + 8 * i * sh.group, o);
      }
      if (has_b) {
        P2 w[4];
        get_columns(c_post, vecs, c, w);
        if (FULL) {
          P2 dz[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            P2 v;
            if (a.gate_dtype == MOE_BF16) {
              v = from_bf16x2(reinterpret_cast<const uint32_t *>(row + src[4].at)[4 * c + k]);
            } else {
              const float2 z = reinterpret_cast<const float2 *>(row + src[4].at)[4 * c + k];
              v = pair(z.x, z.y);
            }
            dz[k] = d[i][k] * b[i].two(k) * w[k] * rs;
            if (sig) {
              const float2 z = split(v);
              const float z0 = sigmoid(z.x), z1 = sigmoid(z.y);
              v = pair(z0, z1);
              dz[k] = dz[k] * pair(z0 * (1.0f - z0), z1 * (1.0f - z1));
            }
            d[i][k] = d[i][k] * v;
          }
          if (g.dgate) {
            if (a.gate_dtype == MOE_BF16)
              store_pairs(static_cast<uint16_t *>(g.dgate) + t * g.ld_dgate + 8 * (c0 + c), dz);
            else
              store_pairs(static_cast<float *>(g.dgate) + t * g.ld_dgate + 8 * (c0 + c), dz);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const P2 p = d[i][k] * b[i].two(k);
          sum_post[i][k] = fma2(p, rs, sum_post[i][k]);
          q2 = fma2(p, w[k], q2);
          d[i][k] = d[i][k] * w[k];
        }
      }
    }
    px += step_x;
    if (!has_b) {
      if (kLate) {
        __syncwarp();
        sync();
        if (T - t > ahead) ring_copy(copies, src, row, full, t + ahead);
      }
      continue;
    }
    // q: the sum of d g w b (token gates: without g)
    float q[1] = {total(q2)};
    if (post || token) {
      group_sum(q, warps, warp, sm.red[group][turn][1], sync);
      if (SPLIT && ahead != kGaveUp && !add_other(q, sm, turn, 1, half_phase, rank, status)) ahead = kGaveUp;
    }
    if (kLate) {
      if (!(post || token)) {
        __syncwarp();
        sync();
      }
      if (T - t > ahead) ring_copy(copies, src, row, full, t + ahead);
    }
    if (token && g.dgate && tid == 0 && rank == 0)
      store1_any(g.dgate, a.gate_dtype, t, (sig ? gate_t * (1.0f - gate_t) : 1.0f) * q[0] * rb);
    if (out_db) {
      // db = rb (g d w - h mean(g d w h)), h = b rb; without a norm g d, whatever b is
      const P2 rb2 = twice(rb), g2 = twice(gate_t), back_b = twice(-rb * (rb * q[0] * gate_t * inv_h));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (tid + i * sh.group >= vecs) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          d[i][k] = d[i][k] * g2;
          if (post) d[i][k] = fma2(b[i].two(k), back_b, d[i][k]) * rb2;
        }
        store_pairs(pb + 8 * i * sh.group, d[i]);
      }
    }
    pb += step_b;
  }
  // the block's part: its groups' sums, in group order, by way of the ring's
  // memory (no copy is in flight: every row that was asked for was waited for)
  float *part = parts + (int64_t)block * 2 * H + 8 * c0;
  float *join = reinterpret_cast<float *>(ring_smem + 2 * cols * 4);
  const bool wanted[2] = {g.dw_pre != nullptr, g.dw_post != nullptr || (a.gate_kind == MOE_GATE_CHANNEL && g.dgate)};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!wanted[k]) continue;
    for (int from = 0; from < sh.groups; ++from) {
      if (sh.groups > 1) __syncthreads();
      if (group != from) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * sh.group;
        if (c >= vecs) continue;
        P2(&sum)[4] = k == kSumPre ? sum_pre[i] : sum_post[i];
        if (from > 0) {
          Raw8<float> before;
          before.load(join + 8 * c);
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[j] = before.two(j) + sum[j];
        }
        store_pairs(from + 1 < sh.groups ? join + 8 * c : part + k * H + 8 * c, sum);
      }
    }
  }
  if (ahead == kGaveUp) let_land();
  if (SPLIT) {                             // the other block may still write into this one's memory
    __syncthreads();
    cluster_sync();
  }
}

// blockIdx.y: which sum.  A block has 128 columns, four to a lane, and a warp
// takes every kPartWarps-th part: a thread's loads (10 for 152 parts) are all
// in flight at once.
constexpr int kPartWarps = 16;

__global__ void __launch_bounds__(32 * kPartWarps) norm_parts_kernel(const moe_norm_args a, const moe_norm_grads g,
                                                                     const float *parts, int n) {
  __shared__ float4 red[kPartWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int H = (int)a.H, which = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  if (which == kSumPre ? g.dw_pre == nullptr : g.dw_post == nullptr && !(channel && g.dgate)) return;
  const int c4 = blockIdx.x * 128 + 4 * lane;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c4 < H) {
    const float *from = parts + (int64_t)which * H + c4;
    for (int p = warp; p < n; p += 10 * kPartWarps) {
      float4 v[10];                        // with a test of each, or the last ones' loads would wait for each other
#pragma unroll
      for (int i = 0; i < 10; ++i) {
        const int at = p + i * kPartWarps;
        v[i] = at < n ? *reinterpret_cast<const float4 *>(from + (int64_t)at * 2 * H) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < 10; ++i) s = make_float4(s.x + v[i].x, s.y + v[i].y, s.z + v[i].z, s.w + v[i].w);
    }
  }
  red[warp][lane] = s;
  const int c = blockIdx.x * 128 + (int)threadIdx.x;
  const bool last = threadIdx.x < 128 && c < H;
  float gv = 1.0f, slope = 1.0f, w = 1.0f;
  if (last && which != kSumPre && channel) {
    gv = load1_any(a.gate, a.gate_dtype, c);
    if (a.gate_sigmoid) {
      gv = sigmoid(gv);
      slope = gv * (1.0f - gv);
    }
    if (a.w_post) w = load1_any(a.w_post, a.w_dtype, c) + a.weight_offset;
  }
  __syncthreads();
  if (!last) return;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPartWarps; ++i) sum += reinterpret_cast<const float *>(red[i])[threadIdx.x];
  if (which == kSumPre) {
    g.dw_pre[c] = sum;
    return;
  }
  if (channel && g.dgate) store1_any(g.dgate, a.gate_dtype, c, sum * w * slope);
  if (g.dw_post) g.dw_post[c] = sum * gv;
}

// ---------------------------------------------------------------- host

bool dtype_ok(int32_t d) { return d == MOE_BF16 || d == MOE_F32; }

// A row tensor that has to be there.
int check_row(const void *p, int64_t ld, int64_t H) {
  if (!p || ld < H) return MOE_ERR_INVALID_ARG;
  if (ld % 8 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  return aligned(p, 16) ? MOE_OK : MOE_ERR_MISALIGNED;
}

int check_norm(const moe_norm_args *a) {
  if (!a || a->struct_size != sizeof(moe_norm_args)) return MOE_ERR_INVALID_ARG;
  if (a->T < 0 || a->H <= 0 || !dtype_ok(a->x_dtype) || !dtype_ok(a->w_dtype) || !(a->eps >= 0.f))
    return MOE_ERR_INVALID_ARG;
  if (a->gate_kind < MOE_GATE_NONE || a->gate_kind > MOE_GATE_FULL || (a->gate_sigmoid != 0 && a->gate_sigmoid != 1))
    return MOE_ERR_INVALID_ARG;
  if (a->H % 8 != 0 || a->H > kMaxH || a->T > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->T == 0) return MOE_OK;        // row tensors may be null
  if ((a->gate_kind != MOE_GATE_NONE) != (a->gate != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!a->b && (a->gate || a->w_post || !a->w_pre)) return MOE_ERR_INVALID_ARG;
  if (a->gate && !dtype_ok(a->gate_dtype)) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->w_post, 16) || !aligned(a->w_pre, 16)) return MOE_ERR_MISALIGNED;
  if (a->gate && !aligned(a->gate, a->gate_kind == MOE_GATE_TOKEN ? (a->gate_dtype == MOE_F32 ? 4 : 2) : 16))
    return MOE_ERR_MISALIGNED;
  int rc = check_row(a->x, a->ldx, a->H);
  if (rc == MOE_OK && a->b) rc = check_row(a->b, a->ldb, a->H);
  if (rc == MOE_OK && a->gate_kind == MOE_GATE_FULL) rc = check_row(a->gate, a->ld_gate, a->H);
  return rc;
}

// The most shared memory that a block's ring and column constants may have.
constexpr int kMaxRingBytes = 208 * 1024;
constexpr int kMaxRingH = 8192;

struct RingLaunch {
  RingShape shape;
  int rows, smem;             // rows: blocks, or clusters of two
};

// Columns of a row that a block has.
bool is_split(int64_t H) { return H > kMaxRingH; }
int block_columns(int64_t H) { return (int)(is_split(H) ? 8 * ceil_div(H, 16) : H); }

// Rows of up to 4096 columns share a block where there are `many`, more than
// SMs; as many blocks per SM as have 512 threads (128 registers each).
void block_shape(int64_t H, bool many, RingShape &s, int &per_sm) {
  s.group = (int)round_up((size_t)ceil_div(block_columns(H), 8 * V), 32);
  s.groups = many ? std::max(1, std::min(kMaxGroups, kThreads / s.group)) : 1;
  per_sm = std::min(4, std::max(1, kThreads / (s.group * s.groups)));
}

// Most blocks of a backward launch (parts in the workspace).
int most_parts(int64_t T, int64_t H) {
  RingShape s;
  int per_sm;
  block_shape(H, true, s, per_sm);
  return (int)std::min<int64_t>(T, 160 * std::max(2, per_sm));
}

// `row` and `constants`: bytes a column.  As many stages as a block's share of
// the shared memory holds, but no more than a group has rows.  Fewer blocks per
// SM where that share would not hold two stages; a block that has the SM for
// itself holds one at least (8192 columns of 12 bytes and 8 of constants: 160 KB).
RingLaunch ring_launch(int64_t T, int64_t H, int row, int constants) {
  RingLaunch l{};
  int per_sm, stages;
  const int cols = block_columns(H), sms = num_sms() / (is_split(H) ? 2 : 1);
  block_shape(H, T > num_sms(), l.shape, per_sm);
  for (;; --per_sm) {
    stages = (kMaxRingBytes / per_sm - (per_sm - 1) * 10 * 1024 - constants * cols) / (l.shape.groups * row * cols);
    if (stages >= 2 || per_sm == 1) break;
  }
  l.rows = (int)std::min<int64_t>({ceil_div(T, l.shape.groups), (int64_t)per_sm * sms, most_parts(T, H)});
  l.shape.stages = (int)std::min<int64_t>({kMaxStages, stages, ceil_div(T, (int64_t)l.rows * l.shape.groups)});
  const char *env = getenv("MOE_MXQ_DEBUG_INJECT_WAIT");
  l.shape.inject_wait = env && atoi(env) ? 1 : 0;
  l.smem = std::max(l.shape.stages * l.shape.groups * row * cols, cols * 4) + constants * cols;
  return l;
}

template <typename Kernel>
bool allow_smem(Kernel kernel, std::atomic<uint64_t> &ready) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (ready.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRingBytes) != cudaSuccess) return false;
  ready.fetch_or(bit, std::memory_order_release);
  return true;
}

int gate_column_bytes(const moe_norm_args &a) {
  return a.gate_kind == MOE_GATE_FULL ? (a.gate_dtype == MOE_F32 ? 4 : 2) : 0;
}

template <bool SPLIT, typename Kernel, typename... Args>
int launch_rows(Kernel kernel, std::atomic<uint64_t> &ready, const RingLaunch &l, cudaStream_t st, const Args &...args) {
  if (!allow_smem(kernel, ready)) return MOE_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SPLIT ? 2 * l.rows : l.rows));
  cfg.blockDim = dim3((unsigned)(l.shape.group * l.shape.groups));
  cfg.dynamicSmemBytes = (size_t)l.smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename XT, bool SPLIT>
int forward_rows(const moe_norm_args &a, const RingLaunch &l, cudaStream_t st) {
  static std::atomic<uint64_t> ready[3];
  if (a.gate_kind == MOE_GATE_FULL) return launch_rows<SPLIT>(norm_forward_kernel<XT, true, false, SPLIT>, ready[0], l, st, a, l.shape);
  if (a.b && a.w_post && a.w_pre && a.y)
    return launch_rows<SPLIT>(norm_forward_kernel<XT, false, true, SPLIT>, ready[1], l, st, a, l.shape);
  return launch_rows<SPLIT>(norm_forward_kernel<XT, false, false, SPLIT>, ready[2], l, st, a, l.shape);
}

template <typename XT>
int forward_launch(const moe_norm_args &a, cudaStream_t st) {
  const RingLaunch l = ring_launch(a.T, a.H, (int)sizeof(XT) + (a.b ? 2 : 0) + gate_column_bytes(a), 0);
  return is_split(a.H) ? forward_rows<XT, true>(a, l, st) : forward_rows<XT, false>(a, l, st);
}

template <typename XT, bool SPLIT>
int backward_rows(const moe_norm_args &a, const moe_norm_grads &g, const RingLaunch &l, int *status, float *parts,
                  cudaStream_t st) {
  static std::atomic<uint64_t> ready[3];
  auto run = [&](auto kernel, std::atomic<uint64_t> &r) { return launch_rows<SPLIT>(kernel, r, l, st, a, g, l.shape, status, parts); };
  if (a.gate_kind == MOE_GATE_FULL) return run(norm_backward_kernel<XT, true, false, SPLIT>, ready[0]);
  if (a.b && a.w_post && a.w_pre && g.dy && g.dx && g.db) return run(norm_backward_kernel<XT, false, true, SPLIT>, ready[1]);
  return run(norm_backward_kernel<XT, false, false, SPLIT>, ready[2]);
}

template <typename XT>
int backward_launch(const moe_norm_args &a, const moe_norm_grads &g, cudaStream_t st) {
  int *status = static_cast<int *>(g.workspace);
  float *parts = reinterpret_cast<float *>(static_cast<char *>(g.workspace) + kStatusBytes);
  const int x = (int)sizeof(XT);
  const RingLaunch l = ring_launch(
      a.T, a.H, (a.w_pre ? x + 2 : 0) + (g.dy && x == 2 ? x : 0) + (a.b ? 2 : 0) + gate_column_bytes(a), 8);
  const int rc = is_split(a.H) ? backward_rows<XT, true>(a, g, l, status, parts, st)
                               : backward_rows<XT, false>(a, g, l, status, parts, st);
  if (rc != MOE_OK) return rc;
  const bool gate = a.gate_kind == MOE_GATE_CHANNEL && g.dgate;
  if (!g.dw_pre && !g.dw_post && !gate) return MOE_OK;
  return launch_pdl(norm_parts_kernel, dim3((unsigned)ceil_div(a.H, 128), g.dw_post || gate ? 2 : 1), dim3(32 * kPartWarps), 0, st,
                    a, g, static_cast<const float *>(parts), l.rows);
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" int moe_norm_forward(const moe_norm_args *a, cudaStream_t stream) {
  int rc = check_norm(a);
  if (rc != MOE_OK) return rc;
  if (!aligned(a->status, 4)) return MOE_ERR_MISALIGNED;
  if (a->T == 0)
    return !a->status || cudaMemsetAsync(a->status, 0, 64, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  if ((a->w_pre != nullptr) != (a->n != nullptr) || (!a->b && a->y) || (a->b && !a->y && !a->n)) return MOE_ERR_INVALID_ARG;
  if (a->y && (rc = check_row(a->y, a->ldy, a->H)) != MOE_OK) return rc;
  if (a->n && (rc = check_row(a->n, a->ldn, a->H)) != MOE_OK) return rc;
  return a->x_dtype == MOE_F32 ? forward_launch<float>(*a, stream) : forward_launch<uint16_t>(*a, stream);
}

extern "C" size_t moe_norm_workspace_size(int64_t T, int64_t H) {
  if (T < 0 || H <= 0 || H > kMaxH) return 0;
  return kStatusBytes + round_up((size_t)most_parts(T, H) * 2 * (size_t)H * 4, 256);
}

extern "C" int moe_norm_backward(const moe_norm_args *a, const moe_norm_grads *g, cudaStream_t stream) {
  int rc = check_norm(a);
  if (rc != MOE_OK) return rc;
  if (!g || g->struct_size != sizeof(moe_norm_grads)) return MOE_ERR_INVALID_ARG;
  if (!aligned(g->dw_pre, 16) || !aligned(g->dw_post, 16)) return MOE_ERR_MISALIGNED;
  if (!aligned(g->dgate, a->gate_dtype == MOE_F32 ? 4 : 2)) return MOE_ERR_MISALIGNED;   // stored one by one; a full one below
  if (!g->workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned(g->workspace, 256)) return MOE_ERR_MISALIGNED;
  if (g->workspace_bytes < moe_norm_workspace_size(a->T, a->H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (a->T == 0) {
    const size_t w = (size_t)a->H * 4;
    if (cudaMemsetAsync(g->workspace, 0, 64, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (g->dw_pre && cudaMemsetAsync(g->dw_pre, 0, w, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (g->dw_post && cudaMemsetAsync(g->dw_post, 0, w, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (g->dgate && a->gate_kind == MOE_GATE_CHANNEL &&
        cudaMemsetAsync(g->dgate, 0, a->gate_dtype == MOE_F32 ? w : w / 2, stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if ((a->w_pre != nullptr) != (g->dn != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((g->dw_pre && !a->w_pre) || (g->dw_post && !a->w_post) || (g->db && !a->b) || (g->dgate && !a->gate))
    return MOE_ERR_INVALID_ARG;
  if (g->dy && (rc = check_row(g->dy, g->ld_dy, a->H)) != MOE_OK) return rc;
  if (g->dn && (rc = check_row(g->dn, g->ld_dn, a->H)) != MOE_OK) return rc;
  if (g->dx && (rc = check_row(g->dx, g->ld_dx, a->H)) != MOE_OK) return rc;
  if (g->db && (rc = check_row(g->db, g->ld_db, a->H)) != MOE_OK) return rc;
  if (g->dgate && a->gate_kind == MOE_GATE_FULL && (rc = check_row(g->dgate, g->ld_dgate, a->H)) != MOE_OK) return rc;
  return a->x_dtype == MOE_F32 ? backward_launch<float>(*a, *g, stream) : backward_launch<uint16_t>(*a, *g, stream);
}
