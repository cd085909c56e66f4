// Launches that begin while the kernel before them on the stream still runs.
//
// A kernel that calls let_dependents_start() allows the next launch, when that one is made by
// launch_dependent(), to take SMs as soon as every block of this kernel has started and SMs
// come free: its set-up, or work that does not need this kernel's results, then fills the
// ends of this one.  The dependent kernel calls wait_for_prerequisites() before it touches
// what the other writes, and in any case before it ends, so that whatever follows on the
// stream finds both done.
#pragma once

#include <cuda_runtime.h>

namespace pact {

__device__ __forceinline__ void let_dependents_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_prerequisites() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned threads, size_t smem,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace pact
