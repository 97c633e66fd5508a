// Launches of a call's kernels behind one another, and a kernel's settings made once.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

namespace ssattn {

// The dynamic shared memory of `fn`, set once a device (`done`: a bit a device).
inline cudaError_t allow_smem(const void* fn, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A kernel that waits for the one in front of it by itself (wait_for_previous): it is
// launched while that one still runs, so that the launch takes no time of its own.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*fn)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}
#ifdef __CUDACC__
// Until the kernel in front has ended and what it wrote can be read: before the first
// access to anything that it writes or reads.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// From here on the kernel behind may be launched (its blocks start where there is room).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

}  // namespace ssattn
