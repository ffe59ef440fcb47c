// Powers of two, reciprocals and what is made of them by the hardware's approximations; and
// the lengths of a padded batch.
#pragma once

#include <cstdint>

namespace sanatan {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {  // within 2 ulp; below 2^-126: 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {  // within 1 ulp; above 2^126: 0
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + exp(-x)).
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.0f + ex2(x * -kLog2e)); }

// Tokens of sequence b (lens may be null or out of [0, T]).
__device__ __forceinline__ int length_of(const int64_t* lens, int b, int T) {
  if (lens == nullptr) return T;
  const int64_t n = lens[b];
  return n < 0 ? 0 : (n > T ? T : static_cast<int>(n));
}

}  // namespace sanatan
