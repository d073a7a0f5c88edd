// cluster.cuh -- thread-block clusters: ranks, the cluster barrier and stores into another
// CTA's shared memory.
#pragma once

#include <cstdint>

#include "sm103.cuh"

namespace dspark {

__device__ __forceinline__ uint32_t cluster_cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t cluster_cta_count() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Every thread of every CTA of the cluster; shared-memory writes (remote ones too) before it
// are visible after it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Store two floats at `p` (an address of this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_f32x2(void* p, uint32_t rank, float a, float b) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(there), "f"(a), "f"(b) : "memory");
}

// The same by an asynchronous store, and count their 8 bytes on that CTA's copy of the mbarrier `bar`.
__device__ __forceinline__ void st_async_f32x2(void* p, uint64_t* bar, uint32_t rank, float a,
                                               float b) {
  uint32_t there, bar_there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(bar_there)
               : "r"(smem_addr(bar)), "r"(rank));
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
          there),
      "f"(a), "f"(b), "r"(bar_there)
      : "memory");
}

// Wait for the phase of `bar` with the given parity, whose bytes other CTAs of the cluster
// store.  Gives up (false) after `timeout_ns`.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity,
                                                  uint64_t timeout_ns) {
  uint64_t deadline = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (ok != 0u) return true;
    const uint64_t now = globaltimer_ns();
    if (deadline == 0)
      deadline = now + timeout_ns;
    else if (now > deadline)
      return false;
  }
}

}  // namespace dspark
