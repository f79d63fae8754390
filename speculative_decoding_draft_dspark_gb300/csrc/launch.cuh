// Launches that overlap the tail of the kernel before them on the stream: the
// next kernel's CTAs are scheduled as SMs become free and wait, before they
// touch memory, for the earlier kernel to be complete and visible.
#pragma once

#include <cuda_runtime.h>

namespace dspark {

// At the start of every kernel launched by launch_overlapped, by every thread
// and before its first access to global memory.
__device__ __forceinline__ void wait_for_earlier_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the next kernel's CTAs be scheduled once every CTA of this one has
// started; they wait for this kernel's end all the same.
__device__ __forceinline__ void allow_next_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace dspark
