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
// the MMAs, warp 2 allocates TMEM and zeroes ragged ends, warp 3 hands out wgrad's items, warps 4-11 drain the
// accumulators (two per TMEM lane quadrant: forward / dgrad 64-byte row pieces
// from registers, wgrad boxes of 32 rows x 128 bytes through TMA).  Two accumulators
// alternate, so an item's drain overlaps the next item's MMAs.  Every wait is
// bounded (see moe_get_device_status).
//
// Bounds, and what was measured (N = 4096, K = 7168 where not said):
//   many rows an expert    tensor cores   16 384 rows of one expert: forward 494 to 517 us
//                                         (1.86 to 1.95 PFLOP/s), gradients the same within 3 %
//   few rows an expert     HBM, weights   64 rows over 256 experts of 1024 x 2048: 231 MB in 38.5 us
//                                         (6.0 TB/s)
//   both (64 experts, 16 384 rows, Zipf)  4.4 GB and 1.0 TFLOP in 761 to 806 us in a burst; at the
//                                         power limit, back to back, 870 us
//   wgrad, few rows        HBM, stores    32 experts of 128 rows, BF16: 1.97 GB in 308 us (6.4 TB/s);
//                                         64 of 32 rows, BF16: 522 us (7.3 TB/s); 256 of 31 rows,
//                                         1024 x 2048, float32: 322 us (6.8 TB/s; zeros alone are
//                                         written at 7.5, a copy runs at 6.8)
#include <cuda_bf16.h>

#include <atomic>
#include <cstdlib>
#include <mutex>
#include <type_traits>

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
  static constexpr int kHalfBox = 64 * kBK * 2;        // a 64 x 64 box (M- / N-major operands)
  static constexpr int kFirstEpiWarp = 4;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 32 * (kFirstEpiWarp + kEpiWarps);
  static constexpr int kMaxStages = 6;
  // wgrad: items worked out ahead of the slowest role (two: 331 instead of 310 us
  // for 32 experts of 128 rows, N = 4096, K = 7168 in BF16; four: 16.5 instead of
  // 16.0 for 30 experts of 33 rows, 1000 x 1000, where a pair has six items)
  static constexpr int kClaims = 3;
  static constexpr int kNumBars = 4 * kMaxStages + 6 + 4 * kClaims + 1;
};

// Shared memory of one direction: a ring of slots (stages), staging of the
// output, barriers, tables.
// forward / dgrad: a slot holds, by the item's rows,
//   up to 32:   two reduction blocks (A, A, B, B: 16 + 16 + 2 + 2 KB): such
//               items are bound by HBM, and 192 KB in flight per SM hide its
//               latency;
//   up to 320:  one block (A 16 KB, B 20 KB).
// Six slots: with five, 16 384 rows of one expert (N = 4096, K = 7168) took 539
// instead of 494 us.  The output goes from registers to memory.
// wgrad: one block (A 16 KB, B 16 KB).  It stages its output for TMA stores, a
// 4 KB box per warp: two would cost a stage (32 experts of 128 rows, BF16: 333
// instead of 308 us; 64 of 256 rows, float32: 1220 instead of 1172).
template <int OP>
struct Layout {
  static constexpr bool kW = OP >= kWgrad;
  static constexpr int kSlot = kW ? 32768 : 36864;
  static constexpr int kStages = GP::kMaxStages;
  static constexpr int kEpiBytes = kW ? 4096 : 0;       // per epilogue warp
  static constexpr int kOffEpi = kStages * kSlot;
  static constexpr int kOffBar = kOffEpi + GP::kEpiWarps * kEpiBytes;
  static constexpr int kOffTmemPtr = (kOffBar + 8 * GP::kNumBars + 63) & ~63;
  static constexpr int kOffClaims = kOffTmemPtr + 16;  // wgrad: answers (and one for draining), items
  static constexpr int kOffTab = kOffTmemPtr + 64;     // forward / dgrad: Lists::first[2][E+1]
  static constexpr int kEnd = kW ? kOffClaims + 16 * (GP::kClaims + 1) + 32 * GP::kClaims : kOffTab;
  static constexpr size_t bytes(int E) { return 1024 + kEnd + (kW ? 0 : (size_t)8 * (E + 1)); }
};

// float32 gradients: reduction blocks whose sum the tensor core holds before it
// is added to the item's float32 sum.  The tensor core truncates each addition to its
// accumulator, an error that grows with the length: in norm 2.3e-7 of the result
// for parts of 256 rows, 4.7e-7 for 512, 1.0e-6 for 1024, whatever the number of
// parts, where a float32 product is off by 1e-7 to 5e-7 (64 to 16 384 rows).
// Parts of 256 cost up to 9 % against parts of 1024: N = 4096, K = 7168, 8
// experts of 2048 rows 621 instead of 570 us, 16 of 1024 rows 761 instead of 703,
// 32 of 512 rows 810 instead of 790; one of 16 384 rows 562 instead of 548.
constexpr int kPartBlocks = 4;

constexpr int kSmallB = 2048;       // forward / dgrad: B of one of a slot's two blocks

constexpr long long kLimit = 2000000000LL;              // ~1 s
constexpr long long kInjectedLimit = 20000000LL;        // ~10 ms: the debug wait's budget
constexpr int kMaxExperts = 1024;
static_assert(Layout<kForward>::bytes(kMaxExperts) <= 232448 && Layout<kWgrad>::bytes(kMaxExperts) <= 232448 &&
                  Layout<kWgradF32>::bytes(kMaxExperts) <= 232448,
              "shared memory of one CTA");

struct GMaps {
  CUtensorMap a;        // w (3-D) or dy
  CUtensorMap b[5];     // row operand with boxes of kBoxRows rows; wgrad: b[0] = x in 64 x 64 boxes,
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

constexpr int kBoxRows[5] = {16, 32, 64, 80, 128};
__device__ __forceinline__ int box_of(int rows) {
  return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : rows <= 80 ? 3 : 4;
}
__device__ __forceinline__ int box_rows(int box) { return box < 3 ? 16 << box : box == 3 ? 80 : 128; }

struct GItem {
  int e, m, c;          // expert, pair of 128-row M tiles, wgrad: 256-column N tile
  int row0, rows;       // forward / dgrad: first row and rows of the tile; wgrad: of the expert
  int kb, per;          // reduction blocks, in all and per stage
  bool once;            // forward / dgrad: no other tile reads these weights
  int n, n2;            // N slots (multiples of 32) of the MMA, of a second one for the rows after the first n
};

// forward / dgrad: where the items of a launch lie.  An item is a tile of an
// expert's rows times a 256-wide M tile.  An expert's rows are cut into equal
// tiles of up to 256, or 320 where that saves one: up to 256 fill one accumulator, so that its
// drain overlaps the next item's MMAs; more take both (two MMAs per A tile),
// which costs that overlap but not a second pass over the weights (an expert of
// 264 rows as 256 + 8 took 1.2 times as long).
// Items fall in two lists, each expert-major: those of experts with more than
// one tile, bound by the tensor cores, and those of experts with one, bound by
// HBM where it has few rows.  The lists are merged in proportion, kRun items at
// a time, so that both are busy all along.  Within an expert, groups of kGroup
// tiles are walked tiles first: the items in flight then share rows as well as
// weights in L2 (64 experts, 16 384 rows, skewed, N = 4096, K = 7168: HBM reads
// 4.6 GB instead of 5.2, of which 4.0 are each operand once; 4.4 with the loads'
// hint on weights that one tile reads).
constexpr int kRun = 16;
constexpr int kGroup = 8;

__device__ __forceinline__ int tiles_of(int rows) { return rows <= 320 ? (rows > 0) : rows <= 576 ? 2 : (rows + 255) / 256; }

struct Lists {
  const int32_t *offsets;
  const int *first;      // [2][E+1]: first tile of each expert in the two lists (many, one)
  int E, mt;             // experts, M tiles
  int items0, items1, runs0, runs1;

  __device__ __forceinline__ int total() const { return (runs0 + runs1) * kRun; }
  // The w-th place: false where a list's last run has no item left.
  __device__ __forceinline__ bool at(int w, GItem &it) const {
    int list, i = w;
    if (runs0 == 0 || runs1 == 0) {
      list = runs0 == 0 ? 1 : 0;
    } else {
      const unsigned run = (unsigned)w / kRun, n = (unsigned)(runs0 + runs1), a = (unsigned)runs0;
      unsigned before, upto;                                 // runs of the first list before / up to this one
      if (n < 65536u) {
        before = run * a / n;
        upto = (run + 1) * a / n;
      } else {
        before = (unsigned)((uint64_t)run * a / n);
        upto = (unsigned)((uint64_t)(run + 1) * a / n);
      }
      list = upto > before ? 0 : 1;
      i = (int)(list == 0 ? before : run - before) * kRun + w % kRun;
    }
    if (i >= (list == 0 ? items0 : items1)) return false;
    const int *f = first + list * (E + 1);
    const int tile = i / mt;
    int lo = 0, hi = E;                                      // f[lo] <= tile < f[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (f[mid] <= tile) lo = mid; else hi = mid;
    }
    it.e = lo;
    it.c = 0;
    it.once = list == 1;
    it.m = i - f[lo] * mt;
    it.row0 = __ldg(offsets + lo);
    it.rows = __ldg(offsets + lo + 1) - it.row0;
    if (list == 0) {
      const int tiles = f[lo + 1] - f[lo];
      const int group = it.m / (kGroup * mt), r = it.m - group * (kGroup * mt);
      const int in_group = min(kGroup, tiles - group * kGroup);
      it.m = r / in_group;
      // equal tiles: the first `longer` have a row more
      const int t = group * kGroup + r - it.m * in_group;
      const int size = it.rows / tiles, longer = it.rows - size * tiles;
      it.row0 += t * size + min(t, longer);
      it.rows = size + (t < longer ? 1 : 0);
    }
    it.per = it.rows <= 32 ? 2 : 1;
    it.n = it.rows <= GP::kN ? (it.rows + 31) & ~31 : ((it.rows + 1) / 2 + 31) & ~31;
    it.n2 = it.rows <= GP::kN ? 0 : (it.rows - it.n + 31) & ~31;
    return true;
  }
};

// forward / dgrad: the items at places w, w + step, ... of one pair.
struct Places {
  const GArgs &g;
  const Lists &lists;
  int w, step, total;
  GItem it;

  __device__ __forceinline__ bool more() const { return w < total; }
  __device__ __forceinline__ void find() {
    while (w < total && !lists.at(w, it)) w += step;
  }
  __device__ __forceinline__ void start(bool) {
    it.kb = (g.R + GP::kBK - 1) / GP::kBK;
    find();
  }
  __device__ __forceinline__ void next() {
    w += step;
    find();
  }
};

// wgrad: a launch has a pair of CTAs for each item.  A pair works on the one
// that it was launched for, then on those of pairs that it keeps from being
// launched (claims): a pair that is quicker does more of them, and they are
// begun in order.  Where all SMs only store, a third of them, whole groups of
// neighbours, is a fifth slower: with fixed shares of 2.1 GB they end 60 of 325 us
// after the others (dw's stores alone: 6.7 instead of 7.5 TB/s; 256 experts of 31
// rows, N = 1024, K = 2048, float32: 370 instead of 322 us).  forward and dgrad, whose pairs read
// the same weights from L2 at the same time, are 2 % slower that way.
//
// Warp 3 of the leader claims for both CTAs; each CTA's warp 3 works out the
// item and puts it into a ring that its roles read.
struct Ring {
  uint64_t *claim_full;    // each CTA: an answer has arrived
  uint64_t *claim_empty;   // leader: the other CTA has read it
  uint64_t *claim_drain;
  uint64_t *item_full, *item_empty;
  unsigned char *answer;   // kClaims + 1 of 16 bytes
  int4 *items;             // 2 each: (e, m, c, place), (row0, rows, 0, 0); place -1 after the last
};

struct Claimed {
  const GArgs &g;
  const Ring &ring;
  int w, slot;
  uint32_t phase;
  bool wide;               // the role is a warp, not a thread
  GItem it;

  __device__ __forceinline__ bool more() const { return w >= 0; }
  __device__ __forceinline__ void start(bool warp_wide) {
    w = 0;
    slot = 0;
    phase = 0;
    wide = warp_wide;
    next();
  }
  __device__ __forceinline__ void next() {
    const bool got = mbar_wait_reset(ring.item_full + slot, phase, g.status, kLimit, kWaitArrival, w);
    if (!(wide ? __all_sync(0xffffffffu, got) : got)) {
      w = -1;
      return;
    }
    const int4 a = ring.items[2 * slot], b = ring.items[2 * slot + 1];
    it.e = a.x;
    it.m = a.y;
    it.c = a.z;
    w = a.w;
    it.row0 = b.x;
    it.rows = b.y;
    it.kb = (b.y + GP::kBK - 1) / GP::kBK;
    it.per = 1;
    it.n = min(GP::kN, (g.C - a.z * GP::kN + 31) & ~31);
    it.n2 = 0;
    if (wide) __syncwarp();
    if (!wide || (threadIdx.x & 31) == 0) mbar_arrive(ring.item_empty + slot);
    if (++slot == GP::kClaims) { slot = 0; phase ^= 1; }
  }
};

// Short items are claimed as far ahead as the ring holds them; after one of more
// rows than this (some 20 us) the next is claimed when every role has come to
// it, or pairs would hold items that are far apart in dw (one expert of 16 384
// rows: 504 instead of 567 us, of 8192 rows 264 instead of 293; two experts of
// 4096 rows 270 instead of 264).
constexpr int kLongRows = 4096;

// One thread of each CTA of a pair.
__device__ __forceinline__ void claim_items(const GArgs &g, const Ring &ring, int w, int total, int mt, uint32_t rank) {
  const int ct = (g.C + GP::kN - 1) / GP::kN;
  int *status = g.status;
  int slot = 0;
  uint32_t phase = 0;          // of the slot's answer and item
  bool ok = true, left = true;
  for (;;) {
    // 256-column tiles fastest, so that the items in flight write whole rows of dw
    int4 a = make_int4(0, w / ct, 0, w), b = make_int4(0, 0, 0, 0);
    if (w >= total) a.w = -1;
    if (a.w >= 0) {
      a.z = w - a.y * ct;
      a.x = a.y / mt;
      a.y -= a.x * mt;
      b.x = __ldg(g.offsets + a.x);
      b.y = __ldg(g.offsets + a.x + 1) - b.x;
    }
    ok = mbar_wait_reset(ring.item_empty + slot, phase ^ 1, status, kLimit, kWaitArrival, w);
    if (!ok) break;
    ring.items[2 * slot] = a;
    ring.items[2 * slot + 1] = b;
    mbar_arrive(ring.item_full + slot);
    if (a.w < 0) break;
    if (b.y > kLongRows) {
      ok = mbar_wait_reset(ring.item_empty + slot, phase, status, kLimit, kWaitArrival, w);
      if (!ok) break;
    }
    if (rank == 0) {
      ok = mbar_wait_reset(ring.claim_empty + slot, phase ^ 1, status, kLimit, kWaitArrival, w);
      if (!ok) break;
      mbar_arrive_expect_tx(ring.claim_full + slot, 16);
      mbar_arrive_expect_tx_cluster(mapa_shared(smem_u32(ring.claim_full + slot), 1), 16);
      claim_cluster_pair(ring.answer + 16 * slot, ring.claim_full + slot);
    }
    ok = mbar_wait_reset(ring.claim_full + slot, phase, status, kLimit, kWaitArrival, w, rank != 0);
    if (!ok) break;
    const int cta = claimed_cta(ring.answer + 16 * slot);
    fence_proxy_async_shared();                            // the answer's place is written again by the async proxy
    if (rank != 0) mbar_arrive_done(mapa_shared(smem_u32(ring.claim_empty + slot), 0));
    left = cta >= 0;
    w = left ? cta >> 1 : total;
    if (++slot == GP::kClaims) { slot = 0; phase ^= 1; }
  }
  if (rank != 0) return;
  // after a wait gave up, or with bad offsets (total 0): what is left is claimed
  // and dropped, so that those pairs need not be launched to give up in turn
  for (phase = 0; left && (!ok || total == 0); phase ^= 1) {
    mbar_arrive_expect_tx(ring.claim_drain, 16);
    claim_cluster(ring.answer + 16 * GP::kClaims, ring.claim_drain);
    if (!mbar_wait_reset(ring.claim_drain, phase, status, kLimit, kWaitArrival, slot, false)) return;
    if (claimed_cta(ring.answer + 16 * GP::kClaims) < 0) return;
    fence_proxy_async_shared();
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// forward / dgrad: 32 N slots (`rows` of them rows, from row0) of this warp's
// 32 output columns.  TMEM lanes are output columns; three exchanges between
// lanes (of one value, one word, two words) turn them so that lane l holds
// columns 8 (l / 8) .. + 7 of rows l % 8 + 8 r as 16 bytes, and a store writes
// 64-byte pieces of 8 rows.
__device__ __forceinline__ void store_rows(const uint32_t (&v)[32], int64_t row0, int rows, int col0, const GArgs &g,
                                           int lane) {
  const bool b0 = (lane & 1) != 0, b1 = (lane & 2) != 0, b2 = (lane & 4) != 0;
  uint32_t w[16];                      // rows 2 p + b0, two columns
#pragma unroll
  for (int p = 0; p < 16; ++p) {
    const float a = __uint_as_float(v[2 * p]), b = __uint_as_float(v[2 * p + 1]);
    const float got = __shfl_xor_sync(0xffffffffu, b0 ? a : b, 1);
    w[p] = b0 ? pack_bf16(got, b) : pack_bf16(a, got);
  }
  uint32_t u[8][2];                    // rows 4 q + 2 b1 + b0, four columns
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? w[2 * q] : w[2 * q + 1], 2);
    u[q][0] = b1 ? got : w[2 * q];
    u[q][1] = b1 ? w[2 * q + 1] : got;
  }
  uint16_t *out = reinterpret_cast<uint16_t *>(g.out);
  const int col = col0 + 8 * (lane >> 3);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t got0 = __shfl_xor_sync(0xffffffffu, b2 ? u[2 * r][0] : u[2 * r + 1][0], 4);
    const uint32_t got1 = __shfl_xor_sync(0xffffffffu, b2 ? u[2 * r][1] : u[2 * r + 1][1], 4);
    const uint4 piece = b2 ? make_uint4(got0, got1, u[2 * r + 1][0], u[2 * r + 1][1])
                           : make_uint4(u[2 * r][0], u[2 * r][1], got0, got1);
    const int row = 8 * r + (lane & 7);
    if (row < rows && col < g.M) *reinterpret_cast<uint4 *>(out + (row0 + row) * g.ld_out + col) = piece;
  }
}

// wgrad: a box of 32 rows (TMEM lanes) x 128 bytes (64 BF16 or 32 float32
// columns) of dw, from this lane's values `v`, through swizzled staging to a
// TMA store (`add`: addition), which leaves out what lies outside dw.  dw is
// written once and streams through L2 (evict first: 1024 instead of 1046 us for
// 64 experts of 32 rows, N = 4096, K = 7168 in float32).
template <bool kF32>
__device__ __forceinline__ void store_box(const uint32_t *v, bool add, int row, int col, int e, const CUtensorMap *map,
                                          int lane, unsigned char *buf) {
  if (lane == 0) bulk_wait_read<0>();               // the store before has read the staging
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    uint4 piece;
    if (kF32) {
      piece = make_uint4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_bf16(__uint_as_float(v[8 * p + 2 * j]), __uint_as_float(v[8 * p + 2 * j + 1]));
      piece = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4 *>(buf + lane * 128 + ((p ^ (lane & 7)) << 4)) = piece;
  }
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    if (kF32 && add)
      tma_add_3d(map, buf, col, row, e);
    else
      tma_store_3d(map, buf, col, row, e);
    bulk_commit();
  }
}

// This warp's 32 rows x 128 columns of dw from the accumulator; `none`: no
// rows, zeros.
template <bool kF32>
__device__ __forceinline__ void store_block(uint32_t t_row, bool none, bool add, int row, int col, int e, int C,
                                            const CUtensorMap *map, int lane, unsigned char *buf) {
  constexpr int kCols = kF32 ? 32 : 64;
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
    store_box<kF32>(v, add, row, col + c0, e, map, lane, buf);
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
  unsigned char *const answers = smem + L::kOffClaims;
  const Ring ring{never + 1,
                  never + 1 + GP::kClaims,
                  never + 1 + 4 * GP::kClaims,
                  never + 1 + 2 * GP::kClaims,
                  never + 1 + 3 * GP::kClaims,
                  answers,
                  reinterpret_cast<int4 *>(answers + 16 * (GP::kClaims + 1))};
  uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(smem + L::kOffTmemPtr);
  int *tile_first = reinterpret_cast<int *>(smem + L::kOffTab);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = (int)blockIdx.x >> 1;
  int *status = g.status;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.a);
      for (int i = 0; i < (kW ? 2 : 5); ++i) tma_prefetch_desc(&maps.b[i]);
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
      for (int c = 0; kW && c < GP::kClaims; ++c) {
        mbar_init(ring.claim_full + c, 1);
        mbar_init(ring.claim_empty + c, 1);
        mbar_init(ring.item_full + c, 1);
        // roles: loads, ragged ends, epilogue, the leader's MMAs
        mbar_init(ring.item_empty + c, 2 + GP::kEpiWarps + (rank == 0 ? 1 : 0));
      }
      if (kW) mbar_init(ring.claim_drain, 1);
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
    bad |= o < before || (int64_t)o > g.P;
  }
  bad = __syncthreads_or(bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) report_status(status, kStatusBadIndex);
  const int mt = (g.M + GP::kM - 1) / GP::kM;
  Lists lists{g.offsets, tile_first, g.E, mt, 0, 0, 0, 0};
  int total;
  if (kW) {
    total = g.E * mt * ((g.C + GP::kN - 1) / GP::kN);
  } else {
    if (warp < 2) {
      // warp 0: the list of experts with more than one tile, warp 1: with one;
      // a lane takes a run of experts, so that its loads are all in flight
      int *first = tile_first + warp * (g.E + 1);
      const int per = (g.E + 31) / 32, e0 = min(lane * per, g.E), e1 = min(e0 + per, g.E);
      auto tiles_in_list = [&](int e) {
        const int n = bad ? 0 : tiles_of(__ldg(g.offsets + e + 1) - __ldg(g.offsets + e));
        return (n > 1) == (warp == 0) ? n : 0;
      };
      int sum = 0;
#pragma unroll 8
      for (int e = e0; e < e1; ++e) sum += tiles_in_list(e);
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      int at = upto - sum;
      for (int e = e0; e < e1; ++e) {
        first[e] = at;
        at += tiles_in_list(e);
      }
      if (lane == 31) first[g.E] = upto;
    }
    __syncthreads();
    lists.items0 = tile_first[g.E] * mt;
    lists.items1 = tile_first[2 * g.E + 1] * mt;
    lists.runs0 = (lists.items0 + kRun - 1) / kRun;
    lists.runs1 = (lists.items1 + kRun - 1) / kRun;
    total = lists.total();
  }
  if (bad) total = 0;
  const uint32_t tmem_base = *tmem_ptr;
  auto items = [&] {
    if constexpr (kW)
      return Claimed{g, ring};
    else
      return Places{g, lists, cluster, (int)gridDim.x >> 1, total};
  }();

  if (warp == 0) {
    // ------------------------------------------------------------ loads (both CTAs), one thread
    // The ring's slots are few for the loads' latency, so the way from a free
    // slot to its copies is kept short: everything but the slot is worked out
    // beforehand.
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0, tails = 0, tail_phase = 0;
      bool ok = true;
      const uint32_t full0 = mapa_shared(smem_u32(full), 0);
      items.start(false);
      while (items.more() && ok) {
        const GItem it = items.it;
        if (kW && it.kb == 0) {
          items.next();
          continue;
        }
        const int half = it.n >> 1, half2 = it.n2 >> 1;
        const int box = box_of(half), box2 = box_of(half2);
        const int boxes = half <= 64 ? 1 : 2;                     // wgrad: 64-column boxes of B
        const int b_bytes = kW ? boxes * GP::kHalfBox : box_rows(box) * GP::kBK * 2;
        const int m0 = it.m * GP::kM + (int)rank * 128;
        const CUtensorMap *map_b = &maps.b[box], *map_b2 = &maps.b[box2];
        const int b_row = it.row0 + (int)rank * half, b2_row = it.row0 + it.n + (int)rank * half2;
        const int b_col = it.c * GP::kN + (int)rank * half;
        // weights that one tile reads leave L2 first, and the others' stay (64
        // experts, skewed, N = 4096, K = 7168: 4.39 GB from HBM instead of 4.56,
        // 761 instead of 808 us)
        const uint64_t policy = l2_policy(!kW && it.once);
        // kPer blocks a stage, kTwo: rows in two MMAs
        auto blocks_of = [&](auto per_c, auto two_c) {
          constexpr int kPer = decltype(per_c)::value;
          constexpr bool kTwo = decltype(two_c)::value;
          const uint32_t block_bytes = (uint32_t)(GP::kATile + b_bytes);
          const uint32_t bytes = kPer * block_bytes + (kTwo ? (uint32_t)(box_rows(box2) * GP::kBK * 2) : 0u);
          for (int kb = 0; kb < it.kb; kb += kPer) {
            const bool tail = kW && kb == it.kb - 1 && (it.rows & 15) != 0;
            const bool one = kPer == 2 && kb + 1 >= it.kb;        // the last of an odd number of blocks
            unsigned char *slot = smem + stage * L::kSlot;
            const uint32_t bar = full0 + 8 * (uint32_t)stage;
            if (!mbar_wait_reset(&empty[stage], phase ^ 1, status, kLimit, kWaitProducerEmpty, kb)) return false;
            if (tail) {
              // the ragged block: onto this CTA's own barrier, for warp 2
              if (rank == 0) mbar_arrive(&full[stage]);
              mbar_arrive_expect_tx(&tail_full[stage], bytes);
              for (int j = 0; j < 2; ++j)
                tma_load_2d(slot + j * GP::kHalfBox, &maps.a, &tail_full[stage], m0 + 64 * j, it.row0 + kb * GP::kBK);
              for (int j = 0; j < boxes; ++j)
                tma_load_2d(slot + GP::kATile + j * GP::kHalfBox, &maps.b[0], &tail_full[stage], b_col + 64 * j,
                            it.row0 + kb * GP::kBK);
              tails |= 1u << stage;
              tail_phase ^= 1u << stage;             // parity of the next use of tail_full[stage]
            } else {
              if (rank == 0) mbar_arrive_expect_tx(&full[stage], one ? 2 * block_bytes : 2 * bytes);
              if (kW) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  tma_load_2d_2sm(slot + j * GP::kHalfBox, &maps.a, bar, m0 + 64 * j, it.row0 + kb * GP::kBK);
                tma_load_2d_2sm(slot + GP::kATile, &maps.b[0], bar, b_col, it.row0 + kb * GP::kBK);
                if (boxes == 2)
                  tma_load_2d_2sm(slot + GP::kATile + GP::kHalfBox, &maps.b[0], bar, b_col + 64, it.row0 + kb * GP::kBK);
              } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                  if (i > 0 && one) break;
                  unsigned char *a = slot + i * GP::kATile, *b = slot + kPer * GP::kATile + i * kSmallB;
                  const int k0 = (kb + i) * GP::kBK;
                  if (OP == kForward) {
                    tma_load_3d_2sm(a, &maps.a, bar, k0, m0, it.e, policy);
                  } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) tma_load_3d_2sm(a + j * GP::kHalfBox, &maps.a, bar, m0 + 64 * j, k0, it.e,
                                                                  policy);
                  }
                  tma_load_2d_2sm(b, map_b, bar, k0, b_row);
                  if (kTwo) tma_load_2d_2sm(b + b_bytes, map_b2, bar, k0, b2_row);
                }
              }
            }
            issued |= 1u << stage;
            issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == L::kStages) { stage = 0; phase ^= 1; }
            if (kb == 0) items.next();               // while the first blocks are on their way
          }
          return true;
        };
        using std::integral_constant;
        if (kW || (it.per == 1 && it.n2 == 0))
          ok = blocks_of(integral_constant<int, 1>{}, integral_constant<bool, false>{});
        else if (it.per == 1)
          ok = blocks_of(integral_constant<int, 1>{}, integral_constant<bool, true>{});
        else
          ok = blocks_of(integral_constant<int, 2>{}, integral_constant<bool, false>{});
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
      if (*reinterpret_cast<volatile int *>(status + 1) != 0) {
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader), one thread
    if (rank == 0 && elect_one()) {
      // K-major: 16 K values are 32 bytes of a 128-byte row, 8-row groups 1024
      // bytes apart; M- / N-major: 16 K rows of 128 bytes, 8-row groups 1024
      // bytes apart, 64-wide boxes kHalfBox apart
      constexpr uint64_t kAStep = (OP == kForward ? 32 : 2048) >> 4, kBStep = (kW ? 2048 : 32) >> 4;
      const uint64_t a_desc = make_smem_desc(smem_u32(smem), OP == kForward ? 16 : GP::kHalfBox, 1024, kSwizzle128B);
      const uint64_t b_desc = make_smem_desc(smem_u32(smem), kW ? GP::kHalfBox : 16, 1024, kSwizzle128B);
      int stage = 0, j = 0;
      uint32_t phase = 0, fixed_phase = 0;
      bool ok = true;
      items.start(false);
      while (items.more() && ok) {
        const int w = items.w;
        const GItem it = items.it;
        if (kW && it.kb == 0) {
          items.next();
          continue;
        }
        auto next_acc = [&](int &acc) {                         // the accumulator after the last, drained
          acc = j & 1;
          const uint32_t acc_phase = (uint32_t)(j >> 1) & 1u;
          ++j;
          const bool got = mbar_wait_reset(&tmem_empty[acc], acc_phase ^ 1u, status, kLimit, kWaitMmaTmemEmpty, w);
          tc_fence_after();
          return got;
        };
        int acc, acc2 = 0;
        if (!next_acc(acc) || (it.n2 && !next_acc(acc2))) break;
        if (g.inject_wait == 1 && j <= 2 && w == cluster &&
            !mbar_wait_reset(never, 0, status, kInjectedLimit, kWaitInjected, w))
          break;
        const uint32_t idesc = make_idesc_bf16(GP::kM, (uint32_t)it.n, OP != kForward, kW);
        const uint32_t idesc2 = make_idesc_bf16(GP::kM, (uint32_t)it.n2, OP != kForward, kW);
        const int b2_off = box_rows(box_of(it.n >> 1)) * GP::kBK * 2;
        const int len = kW ? it.rows : g.R;
        int first = 0;                                          // first block of the accumulator's sum
        // kPer blocks a stage, kTwo: rows in two MMAs
        auto blocks_of = [&](auto per_c, auto two_c) {
          constexpr int kPer = decltype(per_c)::value;
          constexpr bool kTwo = decltype(two_c)::value;
          const uint32_t d = tmem_base + (uint32_t)(acc * GP::kN), d2 = tmem_base + (uint32_t)(acc2 * GP::kN);
          uint32_t d_now = d;
          for (int kb = 0; kb < it.kb; kb += kPer) {
            if (OP == kWgradF32 && kb == first + kPartBlocks) { // hand the part over, go on in the other accumulator
              tc_commit_2sm(&tmem_full[acc], 3);
              if (!next_acc(acc)) return false;
              d_now = tmem_base + (uint32_t)(acc * GP::kN);
              first = kb;
            }
            const bool tail = kW && kb == it.kb - 1 && (it.rows & 15) != 0;
            bool got = mbar_wait_reset(&full[stage], phase, status, kLimit, kWaitMmaFull, kb);
            if (tail) {
              got = got &&
                    mbar_wait_reset(&tail_fixed[stage], (fixed_phase >> stage) & 1u, status, kLimit, kWaitMmaFull, kb);
              fixed_phase ^= 1u << stage;
            }
            if (!got) return false;
            {
#pragma unroll
              for (int i = 0; i < kPer; ++i) {
                if (i > 0 && kb + i >= it.kb) break;
                const uint64_t ad = a_desc + (uint64_t)((stage * L::kSlot + i * GP::kATile) >> 4);
                const uint64_t bd = b_desc + (uint64_t)((stage * L::kSlot + kPer * GP::kATile + i * kSmallB) >> 4);
                const uint64_t bd2 = bd + (uint64_t)(b2_off >> 4);
                const int left = len - (kb + i) * GP::kBK;       // reduction values from here on
                if (left > GP::kBK - 16) {
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t more = i > 0 || kk > 0 || kb != first ? 1u : 0u;
                    tc_mma_2sm_f16(d_now, ad + kk * kAStep, bd + kk * kBStep, idesc, more);
                    if (kTwo) tc_mma_2sm_f16(d2, ad + kk * kAStep, bd2 + kk * kBStep, idesc2, more);
                  }
                } else {
                  for (int kk = 0; 16 * kk < left; ++kk) {
                    const uint32_t more = i > 0 || kk > 0 || kb != first ? 1u : 0u;
                    tc_mma_2sm_f16(d_now, ad + kk * kAStep, bd + kk * kBStep, idesc, more);
                    if (kTwo) tc_mma_2sm_f16(d2, ad + kk * kAStep, bd2 + kk * kBStep, idesc2, more);
                  }
                }
              }
              tc_commit_2sm(&empty[stage], 3);
            }
            if (++stage == L::kStages) { stage = 0; phase ^= 1; }
            if (kb == 0) items.next();                         // while the tensor cores are busy
          }
          return true;
        };
        using std::integral_constant;
        if (kW || (it.per == 1 && it.n2 == 0))
          ok = blocks_of(integral_constant<int, 1>{}, integral_constant<bool, false>{});
        else if (it.per == 1)
          ok = blocks_of(integral_constant<int, 1>{}, integral_constant<bool, true>{});
        else
          ok = blocks_of(integral_constant<int, 2>{}, integral_constant<bool, false>{});
        if (!ok) break;
        tc_commit_2sm(&tmem_full[acc], 3);
        if (it.n2) tc_commit_2sm(&tmem_full[acc2], 3);
      }
      tc_commit_2sm(mma_done, 1);
      mbar_wait_reset(mma_done, 0, status, kLimit, kWaitMmaDone, 0, false);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ ragged ends (both CTAs)
    if (kW) {
      int block = 0;                                           // blocks of the items before, modulo the ring
      uint32_t tail_phase = 0;
      items.start(true);
      for (; items.more(); items.next()) {
        const GItem it = items.it;
        if (it.kb > 0 && (it.rows & 15) != 0) {
          const int stage = (block + it.kb - 1) % L::kStages;
          if (!__all_sync(0xffffffffu, mbar_wait_reset(&tail_full[stage], (tail_phase >> stage) & 1u, status, kLimit,
                                                       kWaitMmaFull, items.w)))
            break;
          tail_phase ^= 1u << stage;
          const int rem = it.rows - (it.kb - 1) * GP::kBK;       // 1 .. 63 rows of the block
          const int rows = ((rem + 15) & ~15) - rem;             // rows to zero, 128 bytes in each box
          unsigned char *p = smem + stage * L::kSlot + rem * 128 + lane * 16;
#pragma unroll
          for (int box = 0; box < 4; ++box) {
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
  } else if (warp == 3) {
    if (kW && elect_one()) claim_items(g, ring, cluster, total, mt, rank);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;
    const int ew = warp - GP::kFirstEpiWarp;
    unsigned char *stage_tile = smem + L::kOffEpi + ew * L::kEpiBytes;
    int j = 0;
    items.start(true);
    while (items.more()) {
      const int w = items.w;
      const GItem it = items.it;
      items.next();                                                // before the wait
      const int first = it.m * GP::kM + (int)rank * 128 + 32 * q;  // this warp's M rows
      const int col = it.c * GP::kN + 128 * (ew >> 2);             // wgrad: this warp's columns
      if (kW && it.kb == 0) {                                      // an expert without rows
        if (first < g.M && !g.accumulate)
          store_block<OP == kWgradF32>(0, true, false, first, col, it.e, g.C, &maps.b[1], lane, stage_tile);
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
          for (int c = 0; c < 128; c += 32)
            if (col + c < g.C)
              store_box<true>(reinterpret_cast<uint32_t *>(sum) + c, g.accumulate, first, col + c, it.e, &maps.b[1], lane,
                              stage_tile);
        }
        continue;
      }
      bool got = true;
      for (int part = 0; part < (it.n2 ? 2 : 1); ++part) {
        const int acc = j & 1;
        got = wait_full(acc);
        if (!got) break;
        const uint32_t t_row = t_lane + (uint32_t)(acc * GP::kN);
        if (first < g.M) {
          if (kW) {
            store_block<OP == kWgradF32>(t_row + 128 * (ew >> 2), false, g.accumulate, first, col, it.e, g.C,
                                                    &maps.b[1], lane, stage_tile);
          } else {
            const int row0 = it.row0 + part * it.n, rows = part == 0 ? min(it.rows, it.n) : it.rows - it.n;
            for (int c0 = 32 * (ew >> 2); c0 < rows; c0 += 64) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(t_row + (uint32_t)c0, v);
              tmem_ld_wait();
              store_rows(v, (int64_t)row0 + c0, rows - c0, first, g, lane);
            }
          }
        }
        release(acc);
      }
      if (!got) break;
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
  const int64_t pairs = OP >= kWgrad ? most_items : std::min<int64_t>(num_sms() / 2, most_items);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
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
  for (int i = 0; i < 5; ++i) ok = ok && encode_map(&maps.b[i], in, 2, R, P, 1, ld_in, 0, GP::kBK, kBoxRows[i]);
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
