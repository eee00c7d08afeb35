// gdn_launch.cuh -- launches that overlap the end of the one before them in the stream, and the SMs
// that launches are planned for.
//
// A kernel that is launched with launch_behind may start once every CTA of the launch before it has
// called next_may_start (or ended); what that one wrote is there after wait_for_previous, which
// every CTA calls before it ends, so that the order of later launches holds too.  It saves the
// microsecond or two from the end of one kernel to the start of the next, and the second one's
// set-up.  Launched the usual way, both calls do nothing.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <utility>

#include "gdn_internal.h"

namespace gdn {
namespace {

__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// SMs of the current device, which launches are planned for; 0 where there is none.
inline int current_sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return device_sm_count(dev);
}

// Lets a kernel have `bytes` of dynamic shared memory, which it is told once for every device.
template <auto kernel>
cudaError_t allow_shared(size_t bytes) {
  static std::atomic<unsigned long long> told{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (told.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (err == cudaSuccess) told.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, size_t shared, cudaStream_t stream,
                          Args&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace
}  // namespace gdn
