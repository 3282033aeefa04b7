// follow.cuh - launches that may be set up while the kernel before them on the
// stream still runs (programmatic dependent launch). A kernel launched this way
// calls follow() before its first access to global memory: that waits until
// everything before it on the stream is done and visible, and lets the launch
// after it be set up in turn. What overlaps is the launch itself, barrier and
// TMEM set-up: 2 to 4 us of a call made of several short kernels.
#pragma once

#include <cuda_runtime.h>

namespace dmuon {

__device__ __forceinline__ void follow(bool lead = true) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (lead) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// cluster > 1: thread-block clusters of that many CTAs along x.
template <typename... Params, typename... Args>
cudaError_t launch_follow(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster,
                          const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace dmuon
