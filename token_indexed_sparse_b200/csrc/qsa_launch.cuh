// Launches of kernels that follow one another in a call.
//
// A kernel launched with launch_after may be set up on the GPU while the kernel before it on the
// stream still runs (a programmatic dependency, also inside a captured graph), which takes the launch's
// own 1-2 us off a decode step's chain of short kernels.  Before it reads anything that an earlier
// kernel wrote, it has to wait in after_previous, which returns once the kernel before it has ended and
// its writes can be seen.  That kernel must itself be ordered behind what came before it
// (launched without this, or past its own after_previous), so the order is whole.
//
// What an earlier kernel of the chain writes is not read-only while such a kernel lives, even past the
// wait: it is read by plain loads, through pointers that are not `const __restrict__`, never by __ldg
// (ld.global.nc), which the compiler may move across the wait.
#pragma once

#include <cuda_runtime.h>

namespace qsa {

__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// In the kernel before: the next one may be set up from here on (at its end without this).
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = s;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, static_cast<Params>(args)...);
}

}  // namespace qsa
