// dependent.h -- launches of the expert-layer kernels as programmatic
// dependents, and the start of such a kernel.
#pragma once

#include <atomic>

#include "kernels.h"

namespace nvfp4 {

// The start of a kernel that may run beside the end of the one before it:
// whatever it does before this call touches no global memory, and the next
// kernel may begin the same way (every thread of every CTA calls it, so that
// a finished kernel means a finished predecessor).
__device__ __forceinline__ void grid_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches `func`, which calls grid_begin, so that it may start while the
// preceding kernel on the stream is still running.  cluster: CTAs of a
// cluster, along x.
inline cudaError_t launch_dependent(const void* func, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                    void** args, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, func, args);
}

// Lets `func` use `bytes` of dynamic shared memory on the current device, once
// per device (`allowed`: the devices where it is done, one bit each).
inline cudaError_t allow_smem(const void* func, int bytes, std::atomic<uint64_t>& allowed) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (allowed.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace nvfp4
