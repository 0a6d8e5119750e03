// chain.cuh -- launches of a chain of kernels that depend on one another in
// stream order.
#pragma once

#include <cuda_runtime.h>

namespace fk {

// Kernels of a chain are launched with programmatic stream serialization:
// a kernel may start (set up shared memory, compute addresses) while the one
// before it drains, and waits here before its first read of that kernel's
// results.  The wait returns once the previous grid has completed and its
// writes are visible.
__device__ __forceinline__ void wait_prior_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next grid of the chain start once every block of this one has come
// here or ended; without it that is when every block has ended.
__device__ __forceinline__ void let_next_grid() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
static cudaError_t launch_chained(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                  Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace fk
