// after.cuh -- launches a kernel that follows another one of the same call: it is
// brought up while that one still runs (programmatic dependent launch) and
// begins with wait_for_previous(), which returns once that one has ended and its
// writes are there.
#pragma once

#include <cuda_runtime.h>

namespace msim {

__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The kernel that follows may be brought up as soon as all blocks have said so or ended.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, int block, int smem_bytes, cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem_bytes;
  c.stream = stream;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<const P&>(args)...);
}

}  // namespace msim
