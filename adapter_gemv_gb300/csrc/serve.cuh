// serve.cuh -- device helpers of the serving operators (sm_103a).
#pragma once

#include <atomic>

#include "common.cuh"
#include "serve.h"

namespace mlora {

__device__ __forceinline__ int32_t div_by(const FastDiv &f, int32_t n) {
  const uint32_t u = (uint32_t)n;
  return (int32_t)((uint32_t)((((uint64_t)__umulhi(f.mul, u)) + u) >> f.shift));
}

// ceil(n / d), n >= 0
__device__ __forceinline__ int32_t ceil_by(const FastDiv &f, int32_t n) { return n > 0 ? div_by(f, n - 1) + 1 : 0; }

// Raise the dynamic shared memory that a kernel may be launched with, once per device.
template <auto Kernel>
inline cudaError_t raise_smem(int bytes) {
  static std::atomic<bool> done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

// Launch with programmatic stream serialization: the CTAs may be placed while the kernel before them in
// the stream ends. Every kernel launched this way calls pdl_wait() before its first access to
// global memory, so the order of all reads and writes is the stream's.
template <class... P, class... A>
inline cudaError_t launch_waiting(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster,
                                  cudaStream_t stream, A &&...args) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace mlora
