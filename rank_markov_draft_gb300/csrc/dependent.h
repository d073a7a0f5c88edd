// dependent.h -- launches with attributes: in clusters, and as programmatic dependents of the kernel
// before them on their stream (they start beside its end, and wait for it in griddep_wait).
#pragma once

#include <cuda_runtime.h>

namespace dspark {

struct LaunchShape {
  dim3 grid;
  int threads;
  size_t smem = 0;
  int cluster = 1;
  bool dependent = true;
};

template <typename... Params, typename... Args>
inline cudaError_t launch_kernel(const LaunchShape& shape, cudaStream_t stream, void (*kernel)(Params...),
                                 const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = shape.grid;
  cfg.blockDim = dim3(shape.threads);
  cfg.dynamicSmemBytes = shape.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  if (shape.dependent) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (shape.cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = shape.cluster;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace dspark
