// Launches that follow one another in a sequence of kernels: the next kernel's blocks may start while the
// one before drains, set themselves up, and wait for its results only where they read them. Hides
// the 2-4 us between dependent launches.
#pragma once
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

namespace mt {

// Let the next kernel of the sequence start once every block has come this far.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Until the kernel before has completed and its writes are visible.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Let `kernel` ask for up to `bytes` of dynamic shared memory on the current device. `done` is the kernel's own, a bit a
// device: the attribute costs a microsecond to set, and stays.
template <class... P>
cudaError_t allow_shared(void (*kernel)(P...), int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}
// As below, in clusters of `cluster` blocks.
template <class... P, class... A>
cudaError_t launch_cluster_following(void (*kernel)(P...), dim3 grid, unsigned threads, unsigned cluster, size_t smem,
                                     cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {cluster, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
// Launch `kernel`, which calls wait_for_previous() before it touches what the kernel before it on the
// stream reads or writes.
template <class... P, class... A>
cudaError_t launch_following(void (*kernel)(P...), dim3 grid, dim3 threads, size_t smem, cudaStream_t stream,
                             const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace mt
