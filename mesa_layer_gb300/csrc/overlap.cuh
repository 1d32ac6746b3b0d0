// overlap.cuh -- kernels of one call that begin before the one ahead of them has ended (programmatic dependent launch).
//
// A kernel launched with launch_after may start once every CTA of the kernel ahead has called may_follow (or ended): its
// set-up and its reads of the call's own inputs then run beside that one's tail.  What earlier kernels of the call write
// may be read, and what they read be written, only after ahead_done, which waits for the end of all of them (at least one
// thread of every CTA calls it, so that ends come in order).  A warp with a bounded wait calls it first: the wait's limit
// counts from there.  The first kernel of a call is launched plainly: everything
// before the call has ended when it starts.
#pragma once

#include <cuda_runtime.h>

namespace mesa {

__device__ __forceinline__ void may_follow() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void ahead_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
bool launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess;
}

}  // namespace mesa
