// What the kernels around a layer share besides psa_device.cuh: packed fp32
// products, and a kernel launched ahead of the end of the one it follows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace psa {

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A pair of launches: the first kernel lets the second one's blocks onto the
// SMs as its own leave them; every thread of the second waits, before it
// touches what the first wrote and before it returns, for the first to be
// complete.
__device__ __forceinline__ void let_next_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... A>
cudaError_t launch_behind(void (*kern)(A...), dim3 grid, uint32_t threads, cudaStream_t stream,
                          A... args) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.stream = stream;
  cfg.attrs = &at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace psa
