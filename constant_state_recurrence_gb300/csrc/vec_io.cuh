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

inline bool at_bytes(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace sanatan
