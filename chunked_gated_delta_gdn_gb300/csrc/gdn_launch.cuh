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

template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), unsigned grid, int threads, size_t shared, cudaStream_t stream,
                          Args&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace
}  // namespace gdn
