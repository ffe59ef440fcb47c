// Values of a row in global memory, V at a time, as floats.
#pragma once

#include <cstdint>

#include "sanatan_math.cuh"

namespace sanatan {

template <int BYTES>
struct Raw;
template <>
struct Raw<2> {
  using type = uint16_t;
};
template <>
struct Raw<4> {
  using type = uint32_t;
};
template <>
struct Raw<8> {
  using type = uint2;
};
template <>
struct Raw<16> {
  using type = uint4;
};

// V neighbours, loaded and stored as one word; p is aligned to it.
template <typename E, int V>
struct Vec {
  using type = typename Raw<V * sizeof(E)>::type;
  type raw;
  __device__ __forceinline__ void load(const E* p) { raw = *reinterpret_cast<const type*>(p); }
  __device__ __forceinline__ void get(float (&f)[V]) const {
    const E* e = reinterpret_cast<const E*>(&raw);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = load_as_float(e + j);
  }
  __device__ __forceinline__ void put(const float (&f)[V]) {
    E* e = reinterpret_cast<E*>(&raw);
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = store_from_float<E>(f[j]);
  }
  __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<type*>(p) = raw; }
};

// V neighbouring floats (16 bytes at a time where V allows it).
template <int V>
__device__ __forceinline__ void load_floats(const float* p, float (&f)[V]) {
  constexpr int N = V % 4 == 0 ? 4 : V;
#pragma unroll
  for (int i = 0; i < V; i += N) {
    Vec<float, N> v;
    float g[N];
    v.load(p + i);
    v.get(g);
#pragma unroll
    for (int j = 0; j < N; ++j) f[i + j] = g[j];
  }
}
template <int V>
__device__ __forceinline__ void store_floats(float* p, const float (&f)[V]) {
  constexpr int N = V % 4 == 0 ? 4 : V;
#pragma unroll
  for (int i = 0; i < V; i += N) {
    Vec<float, N> v;
    float g[N];
#pragma unroll
    for (int j = 0; j < N; ++j) g[j] = f[i + j];
    v.put(g);
    v.store(p + i);
  }
}

inline bool at_bytes(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace sanatan
