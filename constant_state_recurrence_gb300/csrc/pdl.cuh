// Programmatic dependent launch, for kernels whose runs are short beside a launch.
#pragma once

#include <cuda_runtime.h>

namespace sanatan {

// For a kernel launched with pdl_attribute(), before its first access to global
// memory: the kernel may start while the one before it in the stream ends, and goes
// on once that one's results are visible; the next one may start as soon as every
// CTA of this one runs.  (Layer-shape gated scan, back to back: 14.3 -> 11.4 us.)
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

inline cudaLaunchAttribute pdl_attribute() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

// kernel<<<grid, threads, shared, st>>>(args...) as such a launch.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, int threads, size_t shared,
                             cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sanatan
