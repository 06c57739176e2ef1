// chain.cuh -- launches that overlap their start with the end of the kernel before them on the stream
// (programmatic dependent launch), for operators whose small calls are short beside a launch.
//
// Such a kernel is resident while the one before it still writes, so nothing that a kernel writes is constant for
// as long as it runs: gains, coefficients and rows are read by ordinary loads behind the wait, never through
// the read-only path, whose contract is that the memory does not change during the grid's whole life.
#pragma once

#include <cuda_runtime.h>

namespace cgtp {

// First thing in a kernel that chain_launch starts: no global memory is touched before the kernels
// before it on the stream have completed, and the next one may be set up from here on.
__device__ __forceinline__ void chain_enter() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t chain_launch(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, Args&&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace cgtp
