// State cache: the constant states of sequences kept in 8 bits.
//
// A sequence's state is `layers` stretches of `inner` float32 values, stretch
// (l, b) at (l B + b) inner; a page holds them as groups of 64 codes (one
// feature row of S a group), the last group of a stretch filled up, with one
// float32 scale s a group:
//   int8:  s = max|x| / 127 rounded to float32; the code is the integer nearest
//          to the exact quotient x / s, ties to even;
//   e4m3:  s = the smallest power of two with max|x| / s <= 448, so that x / s
//          is exact and is rounded once, to e4m3.
// A stored value is code * s, off by at most s / 2 (int8) or 2^-4 of itself
// (e4m3; 2^-10 s where |x| < 2^-6 s).  The denominators z stay in float32: every
// output is divided by Phi(q) . z, and they are 1/64 of the values.
#include <cuda_fp8.h>

#include "sanatan_internal.h"

namespace sanatan {
namespace {

constexpr int kGroup = 64;
constexpr uint32_t kTiny = 0x0d800000u;  // 2^-100: smaller groups are stored as zeros
constexpr uint32_t kLarge = 0x7f000000u; // 2^127: there a code times its scale could overflow

// 16 lanes hold a group, four values each.  A group with a value that is not
// finite, or is 2^127 or more, has the scale NaN, so that it reads back as NaN.
template <int F>
__device__ __forceinline__ uint32_t quantise(const float (&v)[4], float& scale) {
  uint32_t top = 0;  // bit patterns of |v| order like the values, NaN above all
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (top >= kLarge) {
    scale = __uint_as_float(0x7fffffffu);
    return 0;
  }
  if (top < kTiny) {
    scale = 0.0f;
    return 0;
  }
  uint32_t word = 0;
  if (F == SANATAN_CACHE_INT8) {
    scale = __fdiv_rn(__uint_as_float(top), 127.0f);
    const float inv = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // v * inv is within 2e-5 of the quotient, so its nearest integer c is right or
      // one off; the remainder v - c s is exact in one FMA and says which.
      float c = rintf(v[i] * inv);
      const float r = fmaf(-c, scale, v[i]);
      const float two = 2.0f * fabsf(r);
      if (two > scale || (two == scale && (static_cast<int>(c) & 1))) c += copysignf(1.0f, r);
      word |= (static_cast<uint32_t>(static_cast<int>(c)) & 0xffu) << (8 * i);
    }
  } else {
    // 448 = 1.75 * 2^8: the exponent of max|x|, less 8, one more where the
    // mantissa is above 1.75.
    const uint32_t e = (top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    scale = __uint_as_float(e << 23);
    const float inv = __uint_as_float((254u - e) << 23);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    word = lo | (hi << 16);
  }
  return word;
}

template <int F>
__device__ __forceinline__ void restore(uint32_t word, float scale, float (&v)[4]) {
  if (F == SANATAN_CACHE_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = static_cast<float>(static_cast<int>(word << (24 - 8 * i)) >> 24) * scale;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>((word >> (16 * i)) & 0xffffu), __NV_E4M3));
      const float2 f = __half22float2(h);
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  }
}

// The page of sequence b, or -1: none, or a later sequence of the call writes it.
__device__ int64_t page_of(const CacheArgs& a, int b, bool writing) {
  const int64_t p = a.pages[b];
  if (p < 0 || p >= a.num_pages) return -1;
  if (writing)
    for (int i = b + 1; i < a.B; ++i)
      if (a.pages[i] == p) return -1;
  return p;
}

template <int F, bool WRITE>
__global__ void __launch_bounds__(256) cache_kernel(CacheArgs a) {
  const unsigned stretch = blockIdx.x / a.blocks, part = blockIdx.x % a.blocks;
  const int b = static_cast<int>(stretch % a.B), l = static_cast<int>(stretch / a.B);
  const int64_t p = page_of(a, b, WRITE);
  if (p < 0) return;
  const int64_t groups = (a.inner + kGroup - 1) / kGroup;
  const int64_t gi = static_cast<int64_t>(part) * 16 + threadIdx.x / 16;
  const int lane = threadIdx.x % 16;
  const int64_t row = static_cast<int64_t>(l) * a.B + b;  // stretch of the state
  const int64_t at = (p * a.layers + l) * groups + gi;    // group of the cache
  const bool there = gi < groups;
  float* x = a.state + row * a.inner;
  uint32_t* code = reinterpret_cast<uint32_t*>(a.codes) + at * 16 + lane;
  float v[4];
  if (WRITE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = gi * kGroup + lane * 4 + i;
      v[i] = there && k < a.inner ? x[k] : 0.0f;
    }
    float scale;
    const uint32_t word = quantise<F>(v, scale);
    if (there) {
      *code = word;
      if (lane == 0) a.scales[at] = scale;
    }
  } else if (there) {
    restore<F>(*code, a.scales[at], v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = gi * kGroup + lane * 4 + i;
      if (k < a.inner) x[k] = v[i];
    }
  }
  // the values kept in float32, by the same blocks
  for (int64_t k = static_cast<int64_t>(part) * 256 + threadIdx.x; k < a.exact_inner;
       k += static_cast<int64_t>(a.blocks) * 256) {
    float* z = a.exact + row * a.exact_inner + k;
    float* c = a.exact_cache + (p * a.layers + l) * a.exact_inner + k;
    if (WRITE)
      *c = *z;
    else
      *z = *c;
  }
}

template <int F, bool WRITE>
cudaError_t launch(CacheArgs a, cudaStream_t st) {
  cache_kernel<F, WRITE><<<a.blocks * a.layers * a.B, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

int64_t state_cache_blocks(int64_t inner) {
  const int64_t groups = (inner + kGroup - 1) / kGroup;
  return groups < 16 ? 1 : (groups + 15) / 16;
}

cudaError_t state_cache_launch(const CacheArgs& a, bool write, cudaStream_t st) {
  if (a.fmt == SANATAN_CACHE_INT8)
    return write ? launch<SANATAN_CACHE_INT8, true>(a, st) : launch<SANATAN_CACHE_INT8, false>(a, st);
  return write ? launch<SANATAN_CACHE_E4M3, true>(a, st) : launch<SANATAN_CACHE_E4M3, false>(a, st);
}

}  // namespace sanatan
