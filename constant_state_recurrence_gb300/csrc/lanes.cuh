// V neighbouring channels of a thread as float32, in packed pairs where V is even.
#pragma once

#include "f32x2.cuh"
#include "fast_math.cuh"

namespace sanatan {
namespace lanes {

template <int V>
struct Lanes {
  static constexpr int P = V / 2;
  uint64_t p[P];
  __device__ __forceinline__ static Lanes of(float x) {
    Lanes r;
#pragma unroll
    for (int i = 0; i < P; ++i) r.p[i] = f2::pk2(x, x);
    return r;
  }
  __device__ __forceinline__ static Lanes of(const float (&f)[V]) {
    Lanes r;
#pragma unroll
    for (int i = 0; i < P; ++i) r.p[i] = f2::pk2(f[2 * i], f[2 * i + 1]);
    return r;
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < P; ++i) f2::upk2(p[i], f[2 * i], f[2 * i + 1]);
  }
};
template <>
struct Lanes<1> {
  float p;
  __device__ __forceinline__ static Lanes of(float x) { return {x}; }
  __device__ __forceinline__ static Lanes of(const float (&f)[1]) { return {f[0]}; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = p; }
};

template <int V>
__device__ __forceinline__ Lanes<V> fma(const Lanes<V>& a, const Lanes<V>& b, const Lanes<V>& c) {
  Lanes<V> r;
  if constexpr (V == 1) {
    r.p = fmaf(a.p, b.p, c.p);
  } else {
#pragma unroll
    for (int i = 0; i < Lanes<V>::P; ++i) r.p[i] = f2::ffma2(a.p[i], b.p[i], c.p[i]);
  }
  return r;
}
template <int V>
__device__ __forceinline__ Lanes<V> mul(const Lanes<V>& a, const Lanes<V>& b) {
  Lanes<V> r;
  if constexpr (V == 1) {
    r.p = a.p * b.p;
  } else {
#pragma unroll
    for (int i = 0; i < Lanes<V>::P; ++i) r.p[i] = f2::fmul2(a.p[i], b.p[i]);
  }
  return r;
}
template <int V>
__device__ __forceinline__ Lanes<V> sub(const Lanes<V>& a, const Lanes<V>& b) {
  Lanes<V> r;
  if constexpr (V == 1) {
    r.p = a.p - b.p;
  } else {
#pragma unroll
    for (int i = 0; i < Lanes<V>::P; ++i) r.p[i] = f2::fsub2(a.p[i], b.p[i]);
  }
  return r;
}
template <int V>
__device__ __forceinline__ Lanes<V> add(const Lanes<V>& a, const Lanes<V>& b) {
  return fma(a, Lanes<V>::of(1.0f), b);
}

// 1 / (1 + exp(-x)) of each.
template <int V>
__device__ __forceinline__ Lanes<V> sigmoid(const Lanes<V>& x) {
  const Lanes<V> one = Lanes<V>::of(1.0f);
  float f[V];
  mul(x, Lanes<V>::of(-kLog2e)).get(f);
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = ex2(f[j]);
  fma(Lanes<V>::of(f), one, one).get(f);
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = rcp(f[j]);
  return Lanes<V>::of(f);
}

}  // namespace lanes
}  // namespace sanatan
