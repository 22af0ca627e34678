// Launches that follow one another in a sequence of kernels: the next kernel's blocks may start while the
// one before drains, set themselves up, and wait for its results only where they read them. Hides
// the 2-4 us between dependent launches.
#pragma once
#include <cuda_runtime.h>

namespace mt {

// Let the next kernel of the sequence start once every block has come this far.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Until the kernel before has completed and its writes are visible.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch `kernel`, which calls wait_for_previous() before it touches what the kernel before it on the
// stream reads or writes.
template <class... P, class... A>
cudaError_t launch_following(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                             const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace mt
