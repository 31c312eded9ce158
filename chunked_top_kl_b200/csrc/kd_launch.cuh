// Launches that follow one another closely (programmatic dependent launch): a
// kernel launched with launch_next may start while the one before it on the
// stream is still running, as soon as every block of that one has called
// next_may_start, and waits in wait_previous until it has finished and its
// writes are visible.  Each kernel of a chain calls wait_previous before it
// touches anything that a kernel writes, so that the last one's end is the
// end of all.  The first of a call is an ordinary launch, and the last does not
// let another start before its end: what follows the call may be anyone's.
// In a kernel that was launched the ordinary way wait_previous does nothing, but
// next_may_start lets whatever follows start early: a kernel that also runs
// outside a chain must not call it there (GemmArgs::chained).
#pragma once

#include <cuda_runtime.h>

namespace kd {

__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
inline cudaError_t launch_next(void (*kernel)(P...), unsigned grid, unsigned block, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace kd
