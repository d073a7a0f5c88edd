// smem_optin.h -- which kernels a context has opted in to more than 48 KB of dynamic shared memory.
#pragma once

#include <algorithm>
#include <vector>
#include <cuda_runtime_api.h>

namespace dspark {

// The attribute is a kernel's on one device, so each context sets it on its own (the current
// device is the context's): at a kernel's first launch, and again where that failed.
class SmemOptIn {
 public:
  template <typename Kernel>
  cudaError_t operator()(Kernel kernel, int bytes) {
    const void* const fn = reinterpret_cast<const void*>(kernel);
    if (std::find(done_.begin(), done_.end(), fn) != done_.end()) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done_.push_back(fn);
    return e;
  }

 private:
  std::vector<const void*> done_;
};

}  // namespace dspark
