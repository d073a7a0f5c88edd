// async_copy.cuh -- asynchronous copies of the training and verification operators (sm103.cuh has the
// 16-byte one), and an L2 policy.
#pragma once

#include <cstdint>

#include "sm103.cuh"

namespace dspark {

__device__ __forceinline__ void cp_async_4(void* smem_dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(smem_dst)),
               "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}

// The first `bytes` of 16 (or 4) from src, zeros for the rest.
__device__ __forceinline__ void cp_async_16_zfill(void* smem_dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(smem_dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void cp_async_4_zfill(void* smem_dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(smem_dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}

// Wait until at most `kPending` of this thread's committed groups are under way.
template <int kPending>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

}  // namespace dspark
