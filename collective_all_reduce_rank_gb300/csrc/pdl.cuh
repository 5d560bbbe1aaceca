// pdl.cuh -- launches that may start while the kernel before them on the
// stream finishes.  The training operators issue two to a few dozen short
// kernels per call; with the programmatic launch attribute a kernel's CTAs
// are placed, and its barriers and tensor memory set up, under the tail of
// the one before it.  Every kernel launched this way calls pdl_wait() before
// it touches global memory: it returns when all earlier kernels have
// finished and their stores are visible (each of them has waited in turn).
#pragma once

#include <cuda_runtime.h>

#include <utility>

#include "rra_internal.h"

namespace rra {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next kernel's CTAs be placed as this one's leave.  A kernel whose
// CTAs fill the GPU in one wave calls it last: called early, the next one's
// CTAs took what slots were left, unevenly over the SMs (forward and restore
// of 512 rows 18.5 us, called last 16.0).
__device__ __forceinline__ void pdl_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_pdl(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t s, A&&... args) {
  note_grid(grid);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace rra
