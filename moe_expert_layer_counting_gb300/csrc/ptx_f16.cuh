// ptx_f16.cuh -- inline-PTX wrappers of the BF16 products (grouped.cu) beyond
// those of ptx.cuh: 3-D TMA loads of a CTA pair, tcgen05.mma kind::f16 with
// operands of either major, wide TMEM reads, bounded waits of kernels that
// reset their own status words, and claims of clusters not launched yet.
#pragma once
#include <cstdint>
#include <cuda.h>

#include "ptx.cuh"

namespace mxq {

// L2 policies of loads: what is read once leaves first.
__device__ __forceinline__ uint64_t l2_policy(bool once) {
  uint64_t p;
  if (once)
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// TMA tile load into this CTA's shared memory, counted on an mbarrier of
// either CTA of the pair (`bar_cluster`: shared::cluster address).
__device__ __forceinline__ void tma_load_3d_2sm(void *dst, const CUtensorMap *map, uint32_t bar_cluster, int32_t x,
                                                int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// Instruction descriptor of kind::f16: BF16 x BF16 -> float32, M = m, N = n;
// a_mn / b_mn: the operand's M (N) index is the contiguous one in shared
// memory (else its K index is).
__device__ __forceinline__ uint32_t make_idesc_bf16(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
  uint32_t d = 0;
  d |= 1u << 4;                        // D: float32
  d |= 1u << 7;                        // A: BF16
  d |= 1u << 10;                       // B: BF16
  d |= (a_mn ? 1u : 0u) << 15;
  d |= (b_mn ? 1u : 0u) << 16;
  d |= ((n >> 3) & 0x3Fu) << 17;
  d |= ((m >> 4) & 0x1Fu) << 24;
  return d;
}

// D[tmem] (+)= A x B on the tensor cores of both SMs of the pair.
__device__ __forceinline__ void tc_mma_2sm_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Each thread of the warp reads its own TMEM lane, 32 consecutive columns.
__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Orders this thread's generic-proxy shared-memory writes before later
// async-proxy (tensor core) reads of them.
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// TMA tile store / float32 addition of a box in this CTA's shared memory
// (values outside the tensor are left out), one bulk group per commit.
// The store's lines are the first to leave L2.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int32_t x, int32_t y, int32_t z) {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3, %4}], [%1], %5;" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap *map, const void *src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the last N groups of this thread have read their shared memory ...
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// ... or are complete.
template <int N>
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory");
}

// Arrival on an mbarrier of either CTA of the pair by a thread that has no
// memory writes to publish to the other CTA's threads (its TMEM loads are
// complete, tcgen05.wait::ld; or its own shared memory is ordered for the
// tensor core by a proxy fence).  Releasing at cluster scope instead waits for
// every store of the thread to be performed: ~2000 cycles, measured.
__device__ __forceinline__ void mbar_arrive_done(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// As mbar_try_wait, ordered after arrivals of the other CTA of the pair too.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait for a kernel whose first CTA resets the status words when it
// starts (no launch before it does): the abort flag is looked at only after
// kAbortDelay cycles of waiting (~1 ms), when that CTA, the first of the grid
// to be placed, has long done so; a flag left by an earlier call is not seen.
constexpr long long kAbortDelay = 2000000LL;
__device__ __forceinline__ bool mbar_wait_reset(uint64_t *bar, uint32_t parity, int *ws_status, long long limit,
                                                int site, int pos, bool honor_abort = true) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const long long t0 = clock64();
  volatile int *abort_flag = ws_status + 1;
  while (true) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const long long waited = clock64() - t0;
    if (honor_abort && waited > kAbortDelay && *abort_flag) return false;
    if (waited > limit) {
      if (atomicCAS(ws_status + 2, 0, site) == 0) {
        ws_status[3] = (int)blockIdx.x;
        ws_status[4] = pos;
      }
      report_status(ws_status, kStatusTimeout);
      atomicExch(ws_status + 1, 1);
      return false;
    }
  }
}

// ---------------------------------------------------------------- clusters that have not been launched yet
// Asks for one: its launch is cancelled and its place left to the caller, or
// there is none left (nothing is asked after that).  The answer, 16 bytes, is
// written to `answer` and counted on `bar`, of this CTA or (pair) of both CTAs.
__device__ __forceinline__ void claim_cluster(void *answer, uint64_t *bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void claim_cluster_pair(void *answer, uint64_t *bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], "
      "[%1];" ::"r"(smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}
// The index of the claimed cluster's first CTA, or -1.
__device__ __forceinline__ int claimed_cta(const void *answer) {
  int x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
      "ld.shared.b128 a, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "mov.b32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, a;\n\t}"
      : "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return x;
}
// Arms a barrier of either CTA of the pair for `bytes` more.
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t cluster_addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr), "r"(bytes) : "memory");
}

}  // namespace mxq
