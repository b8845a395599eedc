// grouped.cu -- BF16 products grouped by expert with ragged sizes, and their
// gradients, on CTA pairs: one tcgen05.mma.cta_group::2 (M = 256, N up to 256,
// K = 16, kind::f16, float32 accumulators in TMEM) drives two SMs.
//
// With R_e the rows of expert e (offsets[e] <= r < offsets[e+1]):
//   forward  y[r][n]     = sum_k x[r][k] w[e][n][k]      A = w  (K-major),  B = x  (K-major)
//   dgrad    dx[r][k]    = sum_n dy[r][n] w[e][n][k]     A = w  (M-major),  B = dy (K-major)
//   wgrad    dw[e][n][k] = sum_{r in R_e} dy[r][n] x[r][k]  A = dy (M-major), B = x (N-major)
// One kernel: the weight's rows (forward, wgrad) or columns (dgrad) fill the
// M = 256 slots, the ragged rows (wgrad: the weight's columns) the N slots,
// which an item uses in steps of 32, so a short segment costs little.  No
// operand is transposed in memory: the MMA reads either major from the
// 128-byte-swizzled boxes that TMA writes.
//
// Ragged ends.  forward / dgrad: rows past a segment's end are other experts'
// (or no one's); they fill N slots of their own and are not stored.  wgrad
// sums over rows, so the rows of the last 16-row step that lie past the end
// are zeroed in shared memory, in both operands (0 x NaN of a neighbour would
// not be 0): the block's copies land on a barrier of their own CTA, a warp
// zeroes those rows, and the MMA waits for both CTAs' warps.
//
// Roles per CTA (384 threads): warp 0 loads (TMA), warp 1 of the leader issues
// the MMAs, warp 2 allocates TMEM and zeroes ragged ends, warps 4-11 drain the
// accumulators (two per TMEM lane quadrant, each with staging of its own: row
// pieces of 64 bytes, wgrad boxes of 32 rows x 128 bytes for TMA).  Two accumulators
// alternate, so an item's drain overlaps the next item's MMAs.  Every wait is
// bounded (see moe_get_device_status).
#include <cuda_bf16.h>

#include <atomic>
#include <cstdlib>
#include <mutex>

#include "../../include/moe_grouped.h"
#include "host_common.h"
#include "ptx.cuh"
#include "ptx_f16.cuh"

namespace mxq {

namespace {

enum : int { kForward = 0, kDgrad = 1, kWgrad = 2, kWgradF32 = 3 };

struct GP {
  static constexpr int kM = 256;                       // M of a pair's MMA (128 per CTA)
  static constexpr int kN = 256;                       // most N slots of an item
  static constexpr int kBK = 64;                       // reduction values per stage (128 bytes of BF16)
  static constexpr int kATile = 128 * kBK * 2;
  static constexpr int kBTile = (kN / 2) * kBK * 2;
  static constexpr int kHalfBox = 64 * kBK * 2;        // a 64 x 64 box (M- / N-major operands)
  static constexpr int kFirstEpiWarp = 4;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 32 * (kFirstEpiWarp + kEpiWarps);
  static constexpr int kMaxStages = 6;
  static constexpr int kNumBars = 4 * kMaxStages + 6;
};

// Shared memory of one direction.  forward / dgrad stage 2 KB of output per
// epilogue warp.  wgrad stages it for TMA stores: a 4 KB box per warp for BF16
// (two would cost a stage, and the loads' latency counts for more: 348 instead
// of 312 us for 32 experts of 128 rows, N = 4096, K = 7168), two for float32,
// whose twice as many boxes bound the drain (256 experts of 31 rows, N = 1024,
// K = 2048: 381 us with one and six stages).  wgrad's items need no table of
// row tiles, and its offsets are read where they lie.
template <int OP>
struct Layout {
  static constexpr bool kW = OP >= kWgrad;
  static constexpr int kStages = OP == kWgradF32 ? 5 : 6;
  static constexpr int kBoxes = OP == kWgradF32 ? 2 : 1;
  static constexpr int kEpiBytes = kW ? kBoxes * 4096 : 2048;    // per epilogue warp
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kOffA + kStages * GP::kATile;
  static constexpr int kOffEpi = kOffB + kStages * GP::kBTile;
  static constexpr int kOffBar = kOffEpi + GP::kEpiWarps * kEpiBytes;
  static constexpr int kOffTmemPtr = (kOffBar + 8 * GP::kNumBars + 63) & ~63;
  static constexpr int kOffTab = kOffTmemPtr + 64;     // forward / dgrad: off[E+1], Tiles::first[2][E+1]
  static constexpr size_t bytes(int E) { return 1024 + kOffTab + (kW ? 0 : (size_t)12 * (E + 1)); }
};

// float32 gradients: reduction blocks whose sum the tensor core holds before it
// is added to the item's float32 sum.  The tensor core truncates each addition to its
// accumulator, an error that grows with the length (1e-9 of the result per
// row, measured); past 1024 rows it would pass float32's own.
constexpr int kPartBlocks = 16;

constexpr long long kLimit = 2000000000LL;              // ~1 s
constexpr long long kInjectedLimit = 20000000LL;        // ~10 ms: the debug wait's budget
constexpr int kMaxExperts = 1024;
static_assert(Layout<kForward>::bytes(kMaxExperts) <= 232448 && Layout<kWgrad>::bytes(kMaxExperts) <= 232448 &&
                  Layout<kWgradF32>::bytes(kMaxExperts) <= 232448,
              "shared memory of one CTA");

struct GMaps {
  CUtensorMap a;        // w (3-D) or dy
  CUtensorMap b[4];     // row operand with boxes of 16, 32, 64, 128 rows; wgrad: b[0] = x in 64 x 64 boxes,
                        // b[1] = dw in boxes of 32 rows x 128 bytes
};

struct GArgs {
  const int32_t *offsets;
  int64_t P;
  int E;
  int M, R, C;          // M extent, reduction length (forward, dgrad), N extent (wgrad)
  int64_t ld_out;       // forward / dgrad: row stride of the output
  void *out;
  int accumulate;       // wgrad in float32
  int inject_wait;
  int *status;
};

struct GItem {
  int e, m, c;          // expert, pair of 128-row M tiles, wgrad: 256-column N tile
  int row0, rows;       // forward / dgrad: first row and rows of the tile; wgrad: of the expert
  int kb;               // reduction blocks
  uint32_t n_mma;       // N slots of the MMA (a multiple of 32)
};

// The items w, w + step, ... of one cluster, in order.  forward / dgrad: row
// tiles in the order of Tiles, the M tiles of a row tile fastest.  wgrad:
// expert-major, then 256-row tiles, 256-column tiles fastest (so that the items
// in flight write whole rows of dw), advanced without divisions.
//
// Row tiles fall in two lists, each expert-major: those of experts with more
// than one tile, bound by the tensor cores (their weights come from L2 after
// the first tile), and those of experts with one, bound by HBM where it has few
// rows.  The lists are merged in proportion, so that both are busy all along.
struct Tiles {
  const int *off;        // [E+1]
  const int *first;      // [2][E+1]: first tile of each expert in the two lists (many, one)
  int E, n[2];

  __device__ __forceinline__ int total() const { return n[0] + n[1]; }
  // Expert, first row and rows of the t-th tile.
  __device__ __forceinline__ void at(int t, int &e, int &row0, int &rows) const {
    const unsigned nt = (unsigned)total(), na = (unsigned)n[0];
    unsigned before, upto;                                   // tiles of the first list before / up to t
    if (nt < 65536u) {
      before = (unsigned)t * na / nt;
      upto = ((unsigned)t + 1) * na / nt;
    } else {
      before = (unsigned)((uint64_t)t * na / nt);
      upto = (unsigned)(((uint64_t)t + 1) * na / nt);
    }
    const bool many = upto > before;
    const int i = many ? (int)before : t - (int)before;
    const int *f = first + (many ? 0 : E + 1);
    int lo = 0, hi = E;                                      // f[lo] <= i < f[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (f[mid] <= i) lo = mid; else hi = mid;
    }
    e = lo;
    row0 = off[lo] + (i - f[lo]) * GP::kN;
    rows = min(GP::kN, off[lo + 1] - row0);
  }
};

template <int OP>
struct Items {
  static constexpr bool kW = OP >= kWgrad;
  const GArgs &g;
  const Tiles &tiles;         // forward / dgrad
  int mt, ct;
  int w, step, total;
  int e, m, c;                // wgrad: of w
  int dm, dc;                 // wgrad: step in (m, c)

  __device__ __forceinline__ Items(const GArgs &g, const Tiles &tiles, int first, int step, int total)
      : g(g), tiles(tiles), mt((g.M + GP::kM - 1) / GP::kM), ct((g.C + GP::kN - 1) / GP::kN), w(first),
        step(step), total(total), e(0), m(0), c(0), dm(0), dc(0) {
    if (kW) {
      m = w / ct;
      c = w - m * ct;
      dm = step / ct;
      dc = step - dm * ct;
      e = m / mt;
      m -= e * mt;
    }
  }
  __device__ __forceinline__ bool more() const { return w < total; }
  __device__ __forceinline__ void next() {
    w += step;
    if (kW) {
      c += dc;
      m += dm;
      if (c >= ct) { c -= ct; ++m; }
      while (m >= mt) { m -= mt; ++e; }
    }
  }
  __device__ __forceinline__ GItem get() const {
    GItem it;
    if (kW) {
      it.e = e;
      it.m = m;
      it.c = c;
      it.row0 = __ldg(g.offsets + e);
      it.rows = __ldg(g.offsets + e + 1) - it.row0;
      it.kb = (it.rows + GP::kBK - 1) / GP::kBK;
      it.n_mma = (uint32_t)min(GP::kN, (g.C - c * GP::kN + 31) & ~31);
    } else {
      const int t = w / mt;
      it.m = w - t * mt;
      it.c = 0;
      tiles.at(t, it.e, it.row0, it.rows);
      it.kb = (g.R + GP::kBK - 1) / GP::kBK;
      it.n_mma = (uint32_t)((it.rows + 31) & ~31);
    }
    return it;
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// forward / dgrad: 32 N slots (rows c0 .. c0 + 31 of the item) of this warp's
// 32 output columns: TMEM lanes are output columns, so lanes l and l ^ 1 swap
// one value of each slot pair, which gives packed column pairs; staged as
// [row][32 columns], stored as one 64-byte piece per row.
__device__ __forceinline__ void store_rows(const uint32_t (&v)[32], int c0, int col0, const GItem &it, const GArgs &g,
                                           int lane, uint32_t *stage) {
  const bool odd = (lane & 1) != 0;
#pragma unroll
  for (int t = 0; t < 32; t += 2) {
    const float a = __uint_as_float(v[t]), b = __uint_as_float(v[t + 1]);
    const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
    stage[(t + (odd ? 1 : 0)) * 16 + (lane >> 1)] = odd ? pack_bf16(got, b) : pack_bf16(a, got);
  }
  __syncwarp();
  uint16_t *out = reinterpret_cast<uint16_t *>(g.out);
  const int col = col0 + 8 * (lane & 3);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    const uint4 piece = *reinterpret_cast<const uint4 *>(stage + r * 16 + 4 * (lane & 3));
    if (c0 + r < it.rows && col < g.M)
      *reinterpret_cast<uint4 *>(out + (int64_t)(it.row0 + c0 + r) * g.ld_out + col) = piece;
  }
  __syncwarp();
}

// wgrad: BOXES boxes of 32 rows (TMEM lanes) x 128 bytes (64 BF16 or 32 float32
// columns) of dw, from this lane's values `v`, through swizzled staging to a
// TMA store (`add`: addition), which leaves out what lies outside dw.  dw is
// written once and streams through L2 (evict first: 1227 instead of 1305 us for
// 64 experts of 32 rows, N = 4096, K = 7168 in float32).
template <bool kF32, int BOXES>
__device__ __forceinline__ void store_boxes(const uint32_t *v, bool add, int row, int col, int e, int C,
                                            const CUtensorMap *map, int lane, unsigned char *buf) {
  constexpr int kCols = kF32 ? 32 : 64;
  if (lane == 0) bulk_wait_read<0>();               // the stores before have read the staging
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 8 * BOXES; ++p) {
    uint4 piece;
    if (kF32) {
      piece = make_uint4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_bf16(__uint_as_float(v[8 * p + 2 * j]), __uint_as_float(v[8 * p + 2 * j + 1]));
      piece = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4 *>(buf + (p >> 3) * 4096 + lane * 128 + (((p & 7) ^ (lane & 7)) << 4)) = piece;
  }
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
#pragma unroll
    for (int b = 0; b < BOXES; ++b) {
      if (col + b * kCols >= C) break;
      if (kF32 && add)
        tma_add_3d(map, buf + b * 4096, col + b * kCols, row, e);
      else
        tma_store_3d(map, buf + b * 4096, col + b * kCols, row, e);
    }
    bulk_commit();
  }
}

// This warp's 32 rows x 128 columns of dw from the accumulator; `none`: no
// rows, zeros.
template <bool kF32, int BOXES>
__device__ __forceinline__ void store_block(uint32_t t_row, bool none, bool add, int row, int col, int e, int C,
                                            const CUtensorMap *map, int lane, unsigned char *buf) {
  constexpr int kCols = (kF32 ? 32 : 64) * BOXES;
#pragma unroll
  for (int c0 = 0; c0 < 128; c0 += kCols) {
    if (col + c0 >= C) break;
    uint32_t v[kCols];
    if (none) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[i] = 0;
    } else {
#pragma unroll
      for (int h = 0; h < kCols; h += 32)
        tmem_ld_32x32b_x32(t_row + (uint32_t)(c0 + h), *reinterpret_cast<uint32_t(*)[32]>(v + h));
      tmem_ld_wait();
    }
    store_boxes<kF32, BOXES>(v, add, row, col + c0, e, C, map, lane, buf);
  }
}

template <int OP>
__global__ void __launch_bounds__(GP::kThreads, 1) grouped_kernel(const __grid_constant__ GMaps maps, const GArgs g) {
  using L = Layout<OP>;
  constexpr bool kW = L::kW;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint64_t *full = bars;                               // leader: both CTAs' copies of a stage
  uint64_t *empty = full + L::kStages;                // each CTA: stage consumed
  uint64_t *tail_full = empty + L::kStages;           // each CTA: its own copies of a ragged block
  uint64_t *tail_fixed = tail_full + L::kStages;      // leader: both CTAs zeroed the block's end
  uint64_t *tmem_full = tail_fixed + L::kStages;      // each CTA: accumulator ready
  uint64_t *tmem_empty = tmem_full + 2;                // leader: both CTAs drained the accumulator
  uint64_t *mma_done = tmem_empty + 2;
  uint64_t *never = mma_done + 1;
  uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(smem + L::kOffTmemPtr);
  int *off = reinterpret_cast<int *>(smem + L::kOffTab);
  int *tile_first = off + g.E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = (int)blockIdx.x >> 1, nclusters = (int)gridDim.x >> 1;
  int *status = g.status;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.a);
      for (int i = 0; i < (kW ? 2 : 4); ++i) tma_prefetch_desc(&maps.b[i]);
    }
  } else if (warp == 2) {
    if (lane == 0) {
      for (int s = 0; s < L::kStages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
        mbar_init(&tail_full[s], 1);
        mbar_init(&tail_fixed[s], 2);
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
  if (blockIdx.x == 0 && threadIdx.x < 16) status[threadIdx.x] = 0;
  int bad = 0;
  for (int e = threadIdx.x; e <= g.E; e += GP::kThreads) {
    const int o = __ldg(g.offsets + e);
    const int before = e > 0 ? __ldg(g.offsets + e - 1) : 0;
    if (!kW) off[e] = o;
    bad |= o < before || (int64_t)o > g.P;
  }
  bad = __syncthreads_or(bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) report_status(status, kStatusBadIndex);
  const int mt = (g.M + GP::kM - 1) / GP::kM;
  Tiles tiles{off, tile_first, g.E, {0, 0}};
  int total;
  if (kW) {
    total = g.E * mt * ((g.C + GP::kN - 1) / GP::kN);
  } else {
    if (warp < 2) {                      // warp 0: the list of experts with more than one tile, warp 1: with one
      int *first = tile_first + warp * (g.E + 1);
      int base = 0;
      for (int e0 = 0; e0 < g.E; e0 += 32) {
        const int e = e0 + lane;
        int n = !bad && e < g.E ? (off[e + 1] - off[e] + GP::kN - 1) / GP::kN : 0;
        if ((n > 1) != (warp == 0)) n = 0;
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += up;
        }
        if (e < g.E) first[e] = base + s - n;
        base += __shfl_sync(0xffffffffu, s, 31);
      }
      if (lane == 0) first[g.E] = base;
    }
    __syncthreads();
    tiles.n[0] = tile_first[g.E];
    tiles.n[1] = tile_first[2 * g.E + 1];
    total = tiles.total() * mt;
  }
  if (bad) total = 0;
  const uint32_t tmem_base = *tmem_ptr;
  Items<OP> items(g, tiles, cluster, nclusters, total);

  if (warp == 0) {
    // ------------------------------------------------------------ loads (both CTAs)
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0, tails = 0, tail_phase = 0;
    bool ok = true;
    for (; items.more() && ok; items.next()) {
      const GItem it = items.get();
      const int half = (int)it.n_mma >> 1;
      const int box = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
      const int boxes = half <= 64 ? 1 : 2;                       // wgrad: 64-column boxes of B
      const uint32_t bytes = GP::kATile + (kW ? boxes * GP::kHalfBox : (16 << box) * GP::kBK * 2);
      const int m0 = it.m * GP::kM + (int)rank * 128;
      for (int kb = 0; kb < it.kb; ++kb) {
        if (!__all_sync(0xffffffffu,
                        mbar_wait_reset(&empty[stage], phase ^ 1, status, kLimit, kWaitProducerEmpty, kb))) {
          ok = false;
          break;
        }
        const bool tail = kW && kb == it.kb - 1 && (it.rows & 15) != 0;
        if (lane == 0) {
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          unsigned char *a = smem + L::kOffA + stage * GP::kATile, *b = smem + L::kOffB + stage * GP::kBTile;
          if (tail) {
            // the ragged block: onto this CTA's own barrier, for warp 2
            if (rank == 0) mbar_arrive(&full[stage]);
            mbar_arrive_expect_tx(&tail_full[stage], bytes);
            for (int j = 0; j < 2; ++j)
              tma_load_2d(a + j * GP::kHalfBox, &maps.a, &tail_full[stage], m0 + 64 * j, it.row0 + kb * GP::kBK);
            for (int j = 0; j < boxes; ++j)
              tma_load_2d(b + j * GP::kHalfBox, &maps.b[0], &tail_full[stage],
                          it.c * GP::kN + (int)rank * half + 64 * j, it.row0 + kb * GP::kBK);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
            if (OP == kForward) {
              tma_load_3d_2sm(a, &maps.a, bar, kb * GP::kBK, m0, it.e);
            } else if (OP == kDgrad) {
              for (int j = 0; j < 2; ++j)
                tma_load_3d_2sm(a + j * GP::kHalfBox, &maps.a, bar, m0 + 64 * j, kb * GP::kBK, it.e);
            } else {
              for (int j = 0; j < 2; ++j)
                tma_load_2d_2sm(a + j * GP::kHalfBox, &maps.a, bar, m0 + 64 * j, it.row0 + kb * GP::kBK);
            }
            if (kW) {
              for (int j = 0; j < boxes; ++j)
                tma_load_2d_2sm(b + j * GP::kHalfBox, &maps.b[0], bar, it.c * GP::kN + (int)rank * half + 64 * j,
                                it.row0 + kb * GP::kBK);
            } else {
              tma_load_2d_2sm(b, &maps.b[box], bar, kb * GP::kBK, it.row0 + (int)rank * half);
            }
          }
        }
        __syncwarp();
        issued |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (tail) {
          tails |= 1u << stage;
          tail_phase ^= 1u << stage;               // parity of the next use of tail_full[stage]
        }
        if (++stage == L::kStages) { stage = 0; phase ^= 1; }
      }
    }
    // no CTA leaves with copies in flight: the leader waits for both CTAs'
    // copies (the final cluster barrier holds the other until then)
    for (int s = 0; s < L::kStages; ++s) {
      if (rank == 0 && (issued & (1u << s)))
        mbar_wait_reset(&full[s], (issued_phase >> s) & 1u, status, kLimit, kWaitProducerDrain, s, false);
      if (tails & (1u << s))
        mbar_wait_reset(&tail_full[s], ((tail_phase >> s) & 1u) ^ 1u, status, kLimit, kWaitProducerDrain, s, false);
    }
    // after a wait gave up the other CTA may have copies in flight for a stage
    // that the leader never armed: give them time to land (~100 us)
    if (lane == 0 && *reinterpret_cast<volatile int *>(status + 1) != 0) {
      const long long t0 = clock64();
      while (clock64() - t0 < 200000) __nanosleep(1000);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0) {
      // K-major: 16 K values are 32 bytes of a 128-byte row, 8-row groups 1024
      // bytes apart; M- / N-major: 16 K rows of 128 bytes, 8-row groups 1024
      // bytes apart, 64-wide boxes kHalfBox apart
      constexpr uint64_t kAStep = (OP == kForward ? 32 : 2048) >> 4, kBStep = (kW ? 2048 : 32) >> 4;
      const uint64_t a_desc =
          make_smem_desc(smem_u32(smem + L::kOffA), OP == kForward ? 16 : GP::kHalfBox, 1024, kSwizzle128B);
      const uint64_t b_desc =
          make_smem_desc(smem_u32(smem + L::kOffB), kW ? GP::kHalfBox : 16, 1024, kSwizzle128B);
      int stage = 0, j = 0;
      uint32_t phase = 0, fixed_phase = 0;
      bool ok = true;
      for (; items.more() && ok; items.next()) {
        const int w = items.w;
        const GItem it = items.get();
        if (kW && it.kb == 0) continue;
        int acc = j & 1;
        uint32_t acc_phase = (uint32_t)(j >> 1) & 1u;
        ++j;
        if (!__all_sync(0xffffffffu, mbar_wait_reset(&tmem_empty[acc], acc_phase ^ 1u, status, kLimit,
                                                     kWaitMmaTmemEmpty, w)))
          break;
        if (g.inject_wait == 1 && j == 1 &&
            !__all_sync(0xffffffffu, mbar_wait_reset(never, 0, status, kInjectedLimit, kWaitInjected, w)))
          break;
        tc_fence_after();
        uint32_t d_tmem = tmem_base + (uint32_t)(acc * GP::kN);
        const uint32_t idesc = make_idesc_bf16(GP::kM, it.n_mma, OP != kForward, kW);
        const int len = kW ? it.rows : g.R;
        int first = 0;                                          // first block of the accumulator's sum
        for (int kb = 0; kb < it.kb; ++kb) {
          if (OP == kWgradF32 && kb == first + kPartBlocks) {   // hand the part over, go on in the other accumulator
            if (elect_one()) tc_commit_2sm(&tmem_full[acc], 3);
            __syncwarp();
            acc = j & 1;
            acc_phase = (uint32_t)(j >> 1) & 1u;
            ++j;
            if (!__all_sync(0xffffffffu, mbar_wait_reset(&tmem_empty[acc], acc_phase ^ 1u, status, kLimit,
                                                         kWaitMmaTmemEmpty, w))) {
              ok = false;
              break;
            }
            tc_fence_after();
            d_tmem = tmem_base + (uint32_t)(acc * GP::kN);
            first = kb;
          }
          const int left = len - kb * GP::kBK;                  // reduction values from here on
          const bool tail = kW && kb == it.kb - 1 && (it.rows & 15) != 0;
          bool got = mbar_wait_reset(&full[stage], phase, status, kLimit, kWaitMmaFull, kb);
          if (tail) {
            got = got && mbar_wait_reset(&tail_fixed[stage], (fixed_phase >> stage) & 1u, status, kLimit, kWaitMmaFull, kb);
            fixed_phase ^= 1u << stage;
          }
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            const uint64_t ad = a_desc + (uint64_t)((stage * GP::kATile) >> 4);
            const uint64_t bd = b_desc + (uint64_t)((stage * GP::kBTile) >> 4);
            if (left > GP::kBK - 16) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc_mma_2sm_f16(d_tmem, ad + kk * kAStep, bd + kk * kBStep, idesc, kb != first || kk != 0 ? 1u : 0u);
            } else {
              for (int kk = 0; 16 * kk < left; ++kk)
                tc_mma_2sm_f16(d_tmem, ad + kk * kAStep, bd + kk * kBStep, idesc, kb != first || kk != 0 ? 1u : 0u);
            }
            tc_commit_2sm(&empty[stage], 3);
          }
          __syncwarp();
          if (++stage == L::kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (elect_one()) tc_commit_2sm(&tmem_full[acc], 3);
        __syncwarp();
      }
      if (elect_one()) tc_commit_2sm(mma_done, 1);
      __syncwarp();
      mbar_wait_reset(mma_done, 0, status, kLimit, kWaitMmaDone, 0, false);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ ragged ends (both CTAs)
    if (kW) {
      int block = 0;                                           // blocks of the items before, modulo the ring
      uint32_t tail_phase = 0;
      for (; items.more(); items.next()) {
        const GItem it = items.get();
        if (it.kb > 0 && (it.rows & 15) != 0) {
          const int stage = (block + it.kb - 1) % L::kStages;
          if (!__all_sync(0xffffffffu, mbar_wait_reset(&tail_full[stage], (tail_phase >> stage) & 1u, status, kLimit,
                                                       kWaitMmaFull, items.w)))
            break;
          tail_phase ^= 1u << stage;
          const int rem = it.rows - (it.kb - 1) * GP::kBK;       // 1 .. 63 rows of the block
          const int rows = ((rem + 15) & ~15) - rem;             // rows to zero, 128 bytes in each box
          unsigned char *p = smem + L::kOffA + stage * GP::kATile + rem * 128 + lane * 16;
#pragma unroll
          for (int box = 0; box < 4; ++box) {
            if (box == 2) p += L::kOffB + stage * GP::kBTile - (L::kOffA + stage * GP::kATile) - 2 * GP::kHalfBox;
            for (int i = lane; i < rows * 8; i += 32) *reinterpret_cast<uint4 *>(p + (i - lane) * 16) = make_uint4(0, 0, 0, 0);
            p += GP::kHalfBox;
          }
          fence_proxy_async_shared();
          __syncwarp();
          // the zeros lie in this SM's shared memory and are ordered before its
          // tensor core's reads by the proxy fence: the arrival itself has
          // nothing to publish (released at cluster scope it took the warp
          // ~2000 cycles an item and held the MMAs up: 378 instead of 312 us
          // for 32 experts of 128 rows, N = 4096, K = 7168)
          if (lane == 0) mbar_arrive_done(mapa_shared(smem_u32(&tail_fixed[stage]), 0));
        }
        block = (block + it.kb) % L::kStages;
      }
    }
  } else if (warp >= GP::kFirstEpiWarp) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;
    const int ew = warp - GP::kFirstEpiWarp;
    unsigned char *stage_tile = smem + L::kOffEpi + ew * L::kEpiBytes;
    int j = 0;
    for (; items.more(); items.next()) {
      const int w = items.w;
      const GItem it = items.get();
      const int first = it.m * GP::kM + (int)rank * 128 + 32 * q;  // this warp's M rows
      const int col = it.c * GP::kN + 128 * (ew >> 2);             // wgrad: this warp's columns
      if (kW && it.kb == 0) {                                      // an expert without rows
        if (first < g.M && !g.accumulate)
          store_block<OP == kWgradF32, L::kBoxes>(0, true, false, first, col, it.e, g.C, &maps.b[1], lane, stage_tile);
        continue;
      }
      const uint32_t t_lane = tmem_base + ((uint32_t)(32 * q) << 16);
      auto wait_full = [&](int acc) {
        const uint32_t acc_phase = (uint32_t)(j >> 1) & 1u;
        ++j;
        const bool got =
            __all_sync(0xffffffffu, mbar_wait_reset(&tmem_full[acc], acc_phase, status, kLimit, kWaitEpiTmemFull, w));
        tc_fence_after();
        return got;
      };
      auto release = [&](int acc) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_done(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
      };
      if (OP == kWgradF32 && it.kb > kPartBlocks) {
        // a long sum: its parts added up in registers, in order
        float sum[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) sum[i] = 0.f;
        bool got = true;
        for (int kb = 0; kb < it.kb; kb += kPartBlocks) {
          const int acc = j & 1;
          got = wait_full(acc);
          if (!got) break;
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(t_lane + (uint32_t)(acc * GP::kN + 128 * (ew >> 2) + c), v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]);
          }
          release(acc);
        }
        if (!got) break;
        if (first < g.M) {
#pragma unroll
          for (int c = 0; c < 128; c += 32 * L::kBoxes)
            if (col + c < g.C)
              store_boxes<true, L::kBoxes>(reinterpret_cast<uint32_t *>(sum) + c, g.accumulate, first, col + c, it.e, g.C,
                                           &maps.b[1], lane, stage_tile);
        }
        continue;
      }
      const int acc = j & 1;
      if (!wait_full(acc)) break;
      const uint32_t t_row = t_lane + (uint32_t)(acc * GP::kN);
      if (first < g.M) {
        if (kW) {
          store_block<OP == kWgradF32, L::kBoxes>(t_row + 128 * (ew >> 2), false, g.accumulate, first, col, it.e, g.C,
                                                  &maps.b[1], lane, stage_tile);
        } else {
          for (int c0 = 32 * (ew >> 2); c0 < it.rows; c0 += 64) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(t_row + (uint32_t)c0, v);
            tmem_ld_wait();
            store_rows(v, c0, first, it, g, lane, reinterpret_cast<uint32_t *>(stage_tile));
          }
        }
      }
      release(acc);
    }
    if (kW && lane == 0) bulk_wait<0>();
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

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

// A BF16 (or float32) tensor of rank 2 or 3 (strides in elements, innermost 1) with boxes
// of box0 x box1 (x 1), 128-byte swizzled; what lies outside reads as zero.
bool encode_map(CUtensorMap *map, const void *base, int rank, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1,
                uint64_t s2, uint32_t box0, uint32_t box1, bool f32 = false) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const uint64_t size = f32 ? 4 : 2;
  const cuuint64_t strides[2] = {s1 * size, s2 * size};
  const cuuint32_t box[3] = {box0, box1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int OP>
int launch_grouped(const GMaps &maps, const GArgs &g, int64_t most_items, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};                // devices whose kernel attribute is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(grouped_kernel<OP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<OP>::bytes(kMaxExperts)) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    ready.fetch_or(bit, std::memory_order_release);
  }
  const int64_t clusters = std::min<int64_t>(num_sms() / 2, most_items);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * clusters));
  cfg.blockDim = dim3(GP::kThreads);
  cfg.dynamicSmemBytes = Layout<OP>::bytes(g.E);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_kernel<OP>, maps, g) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int check_grouped(int64_t P, int64_t N, int64_t K, int32_t E, const void *offsets, const void *workspace,
                  size_t workspace_bytes) {
  if (P < 0 || N <= 0 || K <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (P > 0x7fffffffLL || N > 0x7fffff00LL || K > 0x7fffff00LL || N % 8 != 0 || K % 8 != 0 || E > kMaxExperts)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!offsets || !workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(offsets, 4)) return MOE_ERR_MISALIGNED;
  if (workspace_bytes < moe_grouped_workspace_size(P, N, K, E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return MOE_OK;
}

int check_rows(const void *p, int64_t ld, int64_t cols) {
  if (!p || ld < cols) return MOE_ERR_INVALID_ARG;
  if (ld % 8 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  return aligned(p, 16) ? MOE_OK : MOE_ERR_MISALIGNED;
}

int injected_wait() {
  const char *env = getenv("MOE_MXQ_DEBUG_INJECT_WAIT");
  return env ? atoi(env) : 0;
}

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
  for (int i = 0; i < 4; ++i) ok = ok && encode_map(&maps.b[i], in, 2, R, P, 1, ld_in, 0, GP::kBK, 16u << i);
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
  const int64_t tiles = std::min<int64_t>(P, P / GP::kN + E);      // most row tiles of any offsets
  return launch_grouped<OP>(maps, g, tiles * ceil_div(M, GP::kM), st);
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
