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

#include "pdl.cuh"
#include "sanatan_internal.h"

namespace sanatan {
namespace {

constexpr int kGroup = 64;
constexpr int threads_of(bool write) { return write ? 128 : 256; }
constexpr int kPart = 64;  // groups of a block
constexpr int kAtOnce = 4096;  // sequences of a writing launch, about
constexpr uint32_t kTiny = 0x0d800000u;   // 2^-100: smaller groups are stored as zeros
constexpr uint32_t kLarge = 0x7f000000u;  // 2^127: there a code times its scale could overflow

// The integers nearest to the exact quotients v / scale, ties to even, as bytes.
// fl(v / scale) itself would round a quotient next to a tie to the tie.  v * inv
// lies within 2e-5 of the quotient, so its nearest integer c (the low bits of v inv
// + 1.5 2^23) is right or one off, and the remainder v - c scale, exact in one
// FMA, says which: a remainder of half a scale or more is rare.
__device__ __forceinline__ uint32_t nearest(const float (&v)[4], float scale) {
  constexpr float kMagic = 12582912.0f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  uint32_t bits[4];
  float r[4], most = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = fmaf(v[i], inv, kMagic);
    bits[i] = __float_as_uint(t);
    r[i] = fmaf(kMagic - t, scale, v[i]);
    most = fmaxf(most, fabsf(r[i]));
  }
  if (2.0f * most >= scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float two = 2.0f * fabsf(r[i]);
      if (two > scale || (two == scale && (bits[i] & 1)))
        bits[i] += r[i] > 0.0f ? 1u : 0xffffffffu;
    }
  }
  return __byte_perm(__byte_perm(bits[0], bits[1], 0x0040), __byte_perm(bits[2], bits[3], 0x0040),
                     0x5410);
}

// The scale of a group whose largest magnitude has the bits `top` (2^-100 to 2^127; the
// kernel gives smaller groups the scale 0 and larger ones, or those with a value that
// is not finite, the scale NaN, with codes of 0).
template <int F>
__device__ __forceinline__ float scale_of(uint32_t top) {
  if (F == SANATAN_CACHE_INT8) {
    // top / 127 rounded: with the rounded reciprocal y of 127 and q = fl(top y), the
    // remainder r = top - 127 q is exact and fl(q + r y) is the rounded quotient
    // (Markstein's theorem).
    constexpr float y = 1.0f / 127.0f;
    const float t = __uint_as_float(top), q = t * y;
    return fmaf(fmaf(-127.0f, q, t), y, q);
  }
  // 448 = 1.75 * 2^8: the exponent of max|x|, less 8, one more where the mantissa is
  // above 1.75.
  return __uint_as_float(((top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0)) << 23);
}

template <int F>
__device__ __forceinline__ uint32_t codes_of(const float (&v)[4], float scale) {
  if (F == SANATAN_CACHE_INT8) return nearest(v, scale);
  const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));  // a power of two
  const uint32_t lo =
      __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi =
      __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

template <int F>
__device__ __forceinline__ void restore(uint32_t word, float scale, float (&v)[4]) {
  if (F == SANATAN_CACHE_INT8) {
    const uint32_t up = word ^ 0x80808080u;  // codes + 128, the low byte of 2^23 + code + 128
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = (__uint_as_float(__byte_perm(up, 0x4b000000u, 0x7540 | i)) - 8388736.0f) * scale;
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

// The page of sequence b, or -1: none.
__device__ __forceinline__ int64_t page_of(const CacheArgs& a, int b) {
  const int64_t p = a.pages[b];
  return p >= a.num_pages ? -1 : p;
}

// Whether a later sequence of the launch writes page p of sequence b too.  By all
// threads of a writing block.
__device__ __forceinline__ bool written_later(const CacheArgs& a, int b, int64_t p) {
  constexpr int kThreads = threads_of(true);
  bool later = false;
  for (int i = b + 1 + static_cast<int>(threadIdx.x); i < a.end; i += kThreads)
    later |= a.pages[i] == p;
  return __syncthreads_or(later);
}

// Four values from x on, of which `left` are there (VEC: all or none).
template <bool VEC>
__device__ __forceinline__ void load(const float* x, int left, float (&v)[4]) {
  if (VEC) {
    const float4 f = left > 0 ? __ldcs(reinterpret_cast<const float4*>(x))
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < left ? x[i] : 0.0f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store(float* x, int left, const float (&v)[4]) {
  if (VEC) {
    if (left > 0) *reinterpret_cast<float4*>(x) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) x[i] = v[i];
  }
}

// One part (64 groups, 16 KB of values) of a stretch.  kLanes lanes have a group; lane
// l its words (four values) l, l + kLanes, ..., so that a warp reads whole lines of
// values and whole sectors of codes.  All of a thread's loads are under way before the
// first is used: eight of 16 bytes when writing (VEC: stretches at 16 bytes).  Writing
// takes eight lanes a group (three exchanges for eight values: 168 us where sixteen
// lanes took 184), reading sixteen and twice the threads (whole lines of codes, four
// loads a thread: one sequence in 5.0 us instead of 5.9).
// Bound: bytes.  64 sequences of 144 states (0.9 GB), int8, GB300: written in 168 us,
// 7.0 TB/s, read in 169 us, 7.0 TB/s (a plain copy: 6.8).  Many small states are bound by
// their blocks instead: 9,216 of 768 values (12 groups of the block's 64, 36 MB, 5.3 us at
// the copy rate) are written in 34 us and read in 16.
template <int F, bool WRITE, bool VEC>
__global__ void __launch_bounds__(threads_of(WRITE)) cache_kernel(const CacheArgs a) {
  constexpr int kThreads = threads_of(WRITE);
  constexpr int kLanes = WRITE ? 8 : 16;
  constexpr int kWords = kGroup / 4 / kLanes;   // of a lane
  constexpr int kRows = kThreads / kLanes;      // groups that the block has in hand at a time
  constexpr int kBatch = kPart / kRows;
  const unsigned stretch = blockIdx.x / a.blocks, part = blockIdx.x % a.blocks;
  const unsigned here_b = a.end - a.begin;  // sequences of this launch
  const int b = a.begin + static_cast<int>(stretch % here_b);
  const int l = static_cast<int>(stretch / here_b);
  const int64_t groups = (a.inner + kGroup - 1) / kGroup;
  const int64_t g0 = static_cast<int64_t>(part) * kPart;  // the block's first group
  const int64_t row = static_cast<int64_t>(l) * a.B + b;  // stretch of the state
  const int here = static_cast<int>(min(groups - g0, static_cast<int64_t>(kPart)));
  const int values = static_cast<int>(min(a.inner - g0 * kGroup, int64_t{kPart * kGroup}));
  const int lane = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
  float* x = a.state + row * a.inner + g0 * kGroup;
  wait_for_previous();

  // Before any other load: nothing of a sequence that is left out is read.
  const int64_t p = page_of(a, b);
  if (p < 0) return;
  if (WRITE) {
    float v[kBatch][kWords][4];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int k = (first + u * kRows) * kGroup + 4 * (lane + i * kLanes);
        load<VEC>(x + k, values - k, v[u][i]);
      }
    if (written_later(a, b, p)) return;
    const int64_t page = (p * a.layers + l) * groups + g0;
    uint32_t* codes = reinterpret_cast<uint32_t*>(a.codes) + page * 16;
    float* scales = a.scales + page;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int g = first + u * kRows;
      uint32_t top = 0;  // bit patterns of |v| order like the values, NaN above all
#pragma unroll
      for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(v[u][i][j]) & 0x7fffffffu);
#pragma unroll
      for (int off = kLanes / 2; off > 0; off /= 2)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
      float scale = scale_of<F>(top);
      uint32_t word[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) word[i] = codes_of<F>(v[u][i], scale);
      if (top < kTiny || top >= kLarge) {
        scale = top < kTiny ? 0.0f : __uint_as_float(0x7fffffffu);
#pragma unroll
        for (int i = 0; i < kWords; ++i) word[i] = 0;
      }
      if (g < here) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) codes[g * 16 + lane + i * kLanes] = word[i];
        if (lane == 0) scales[g] = scale;
      }
    }
    for (int64_t k = static_cast<int64_t>(part) * kThreads + threadIdx.x; k < a.exact_inner;
         k += static_cast<int64_t>(a.blocks) * kThreads)
      a.exact_cache[(p * a.layers + l) * a.exact_inner + k] = a.exact[row * a.exact_inner + k];
    return;
  }
  const int64_t page = (p * a.layers + l) * groups + g0;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes) + page * 16;
  const float* scales = a.scales + page;
  uint32_t word[kBatch][kWords];
  float scale[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int g = first + u * kRows;
    if (g < here) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) word[u][i] = codes[g * 16 + lane + i * kLanes];
      scale[u] = scales[g];
    }
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int g = first + u * kRows;
    if (g < here) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int k = g * kGroup + 4 * (lane + i * kLanes);
        float v[4];
        restore<F>(word[u][i], scale[u], v);
        store<VEC>(x + k, values - k, v);
      }
    }
  }
  for (int64_t k = static_cast<int64_t>(part) * kThreads + threadIdx.x; k < a.exact_inner;
       k += static_cast<int64_t>(a.blocks) * kThreads)
    a.exact[row * a.exact_inner + k] = a.exact_cache[(p * a.layers + l) * a.exact_inner + k];
}

template <int F, bool WRITE>
cudaError_t launch(const CacheArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim =
      dim3(a.blocks * static_cast<unsigned>(a.layers) * static_cast<unsigned>(a.end - a.begin));
  cfg.blockDim = dim3(threads_of(WRITE));
  cfg.stream = st;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool vec = a.inner % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0;
  return vec ? cudaLaunchKernelEx(&cfg, cache_kernel<F, WRITE, true>, a)
             : cudaLaunchKernelEx(&cfg, cache_kernel<F, WRITE, false>, a);
}

}  // namespace

int64_t state_cache_blocks(int64_t inner) {
  const int64_t groups = (inner + kGroup - 1) / kGroup;
  return groups < kPart ? 1 : (groups + kPart - 1) / kPart;
}

// Every block of a write looks through the pages of the launch's later sequences, so a
// write of many goes in launches of about kAtOnce sequences (a page that two of them
// write is the later one's, as within one): the work grows with the sequences, not their
// square.  States of 768 values, int8, GB300, from a flushed L2: 9,216 in 40 us and 65,536
// in 253 us (in one launch 43 and 733; in launches of 2,048: 44 and 273, of 8,192: 43 and
// 269).
cudaError_t state_cache_launch(CacheArgs a, bool write, cudaStream_t st) {
  const int64_t all = a.B, parts = (all + kAtOnce / 2) / kAtOnce;
  const int64_t launches = write && parts > 1 ? parts : 1;
  for (int64_t i = 0; i < launches; ++i) {
    a.begin = static_cast<int>(all * i / launches);
    a.end = static_cast<int>(all * (i + 1) / launches);
    const cudaError_t e =
        a.fmt == SANATAN_CACHE_INT8
            ? (write ? launch<SANATAN_CACHE_INT8, true>(a, st)
                     : launch<SANATAN_CACHE_INT8, false>(a, st))
            : (write ? launch<SANATAN_CACHE_E4M3, true>(a, st)
                     : launch<SANATAN_CACHE_E4M3, false>(a, st));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sanatan
