// follow.cuh -- a kernel that follows another one of the same call: launched
// while that one still runs, so that its launch costs nothing, and held back
// by follow() until all of that one's results are there.
#pragma once

#include <cuda_runtime.h>

namespace dsa {

// First statement of a kernel that is launched by launch_after.
__device__ __forceinline__ void follow() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// In the kernel that it follows: from here on (in all CTAs) it may be launched.
__device__ __forceinline__ void launch_followers() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
bool launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, cudaStream_t stream,
                  A... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.stream = stream;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...) == cudaSuccess;
}

}  // namespace dsa
