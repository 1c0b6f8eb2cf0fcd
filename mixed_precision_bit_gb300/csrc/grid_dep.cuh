// Programmatic dependent launch for the multi-kernel calls: a grid launched by
// launch_dependent may start once every block of the grid before it in the stream
// has called grid_trigger (or exited); grid_wait blocks until that grid has
// completed and its memory is visible.  Both are no-ops for a grid launched
// without the attribute.
#pragma once

#include <cuda_runtime.h>

namespace kitty {

__device__ __forceinline__ void grid_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// behind: as a dependent of the grid before it in the stream; else an ordinary launch.
template <class... P, class... A>
inline cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                                 cudaStream_t s, bool behind, const A&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = behind ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&lc, kernel, P(args)...);
  if (e != cudaSuccess) (void)cudaGetLastError();  // reported here, not by a later call
  return e;
}

template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                                    cudaStream_t s, const A&... args) {
  return launch_behind(kernel, grid, threads, smem, s, true, args...);
}

}  // namespace kitty
