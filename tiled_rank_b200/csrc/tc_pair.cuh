// Tensor-core primitives of the experts' products (sm_100a) beside tc.cuh: MMAs
// with both operands in shared memory, issued for one CTA or for a pair of CTAs
// of a cluster (cta_group::2), the pair's commits and TMA loads, and the remote
// mbarrier arrivals between the two CTAs.  CG is the group's number of CTAs.
#pragma once
#include "tc.cuh"

namespace tileq {
namespace tc {

template <int CG>
__device__ __forceinline__ void alloc_cg(uint32_t *slot_smem, uint32_t ncols) {
  if constexpr (CG == 1) {
    alloc(slot_smem, ncols);
    relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(slot_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void dealloc_cg(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 1)
    dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols) : "memory");
}

// Operand tile descriptor, 128-byte swizzle.  `lbo` (bytes) is used by tiles
// whose contiguous dimension is the output's (M or N): the distance between
// 64-element column groups.  Groups of eight 128-byte rows are 1024 bytes apart
// in either orientation.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo) {
  return sdesc_sw128(saddr) & ~(0x3FFFull << 16) | ((uint64_t)(lbo >> 4) << 16);
}

// D[tmem] (+)= A[smem] * B[smem], issued by one thread (of the pair's first CTA).
template <int CG, bool F8>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  static_assert(CG == 1 || !F8, "e4m3 tiles are of one CTA");
  if constexpr (CG == 1 && !F8)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
  else if constexpr (CG == 2 && !F8)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// Arrive on `bar` (of both CTAs of a pair) once this thread's MMAs so far have completed.
template <int CG>
__device__ __forceinline__ void commit_cg(uint64_t *bar) {
  if constexpr (CG == 1)
    commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// The two halves of pdl_wait_and_release.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// ---------------------------------------------------------------- cluster
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
// Address of `p`'s counterpart in CTA `cta` of the cluster.
__device__ __forceinline__ uint32_t map_cta(const void *p, uint32_t cta) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_addr(p)), "r"(cta));
  return a;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr) : "memory");
}
// The arrival publishes nothing of this thread's (the copies it announces report themselves): relaxed, since a
// release at cluster scope makes the thread wait for its earlier accesses, a microsecond in a producer's loop.
__device__ __forceinline__ void arrive_expect_at(uint32_t cluster_addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;\n" ::"r"(cluster_addr),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void store4_at(uint32_t cluster_addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(cluster_addr), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;\n" ::: "memory"); }
// An arrival for tensor-memory reads alone, which wait::ld and tcgen05.fence::before_thread_sync in front of it order
// with what follows the waiting thread's tcgen05.fence::after_thread_sync.  It hands over nothing else.
__device__ __forceinline__ void arrive_relaxed_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr) : "memory");
}
// mbar_wait with a limit of its own, for what takes longer than a step of a pipeline.
__device__ __forceinline__ bool mbar_wait_for(uint64_t *bar, uint32_t parity, int *status, long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > limit) {
      set_status(status, TILEQ_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// The same with cluster-scope acquire: the arrivals may come from another CTA.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, int *status,
                                                  long long limit = kWaitLimitCycles) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (clock64() - t0 > limit) {
      set_status(status, TILEQ_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// ---------------------------------------------------------------- TMA
// Tile loads whose completion is counted on the mbarrier at cluster address
// `bar` (CG == 2: this CTA's or the pair's first CTA's).  No multicast: every
// CTA loads its own tiles into its own shared memory.
template <int CG>
__device__ __forceinline__ void tma_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
        "{%2, %3, %4}], [%5];\n" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

}  // namespace tc
}  // namespace tileq
