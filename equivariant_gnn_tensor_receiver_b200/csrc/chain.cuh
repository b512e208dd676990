// Kernels of one call, launched while the one before them still runs (programmatic
// dependent launch).
//
// A kernel that another of the same call follows calls chain_next() first thing: once all
// its CTAs run, the follower's may take the place of those that have ended.  The follower
// is launched by chain_launch and calls chain_wait() before it reads what the kernel before
// it wrote, or, if it reads none of that, before it ends: so a call's last kernel ends
// after all others, and whatever the stream holds next sees their results.  The last kernel
// of a call does not call chain_next().  (Only kernels are chained: a capture gets no such
// edge behind a memset.)
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace tpc {

__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// All of the kernel before has ended, its writes are visible.  (What it wrote must not be
// read through __restrict__ const pointers: those loads may move above this.)
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
cudaError_t chain_launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid, cfg.blockDim = block, cfg.dynamicSmemBytes = smem, cfg.stream = st;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace tpc
