// Asynchronous copies from global to shared memory, in groups.
#pragma once

#include <cstdint>

namespace sanatan {

// BYTES (4, 8 or 16), both sides aligned to them.
template <int BYTES>
__device__ __forceinline__ void copy_words(void* to, const void* from) {
  const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(from), "n"(BYTES)
                 : "memory");
}
// bytes (4, 8 or 16), or as many zeros where the source is not real (which is not read then).
__device__ __forceinline__ void copy_or_zeros(void* to, const void* from, bool real, int bytes) {
  const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  const int n = real ? bytes : 0;
  if (bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(n)
                 : "memory");
  else if (bytes == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(from), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(from), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

}  // namespace sanatan
