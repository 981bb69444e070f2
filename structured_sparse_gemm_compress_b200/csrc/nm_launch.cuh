// nm_launch.cuh -- kernel launch helpers shared by the translation units.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace nm {

// Launch with programmatic stream serialization, so the kernel's prologue can
// overlap the tail of the previous kernel in the stream (see pdl_wait).
// cluster > 1: launch as clusters of that many CTAs along x (grid a multiple of it).
template <typename Kern, typename... Args>
static cudaError_t launch_pdl(Kern kern, dim3 grid, int threads, int smem, cudaStream_t s, int cluster,
                              const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The dynamic shared-memory opt-in is a per-device property of a kernel: set it
// once per (kernel, device), remembered in a bit mask of device ordinals.
template <typename Kern>
static cudaError_t smem_opt_in(Kern kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

}  // namespace nm
