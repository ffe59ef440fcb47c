// Selective state space scan, per channel d of [B, T, D] with N states (1 .. 128):
//   delta = dt + dt_bias, or log(1 + exp(dt + dt_bias)),
//   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t u_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + skip u_t) z_t / (1 + exp(-z_t))   (without z: no last factor),
// its gradients, with v = dy z / (1 + exp(-z)), a = exp(delta A) and g_{T} = dh_out,
//   dh_t[n] = v_t C_t[n] + g_{t+1}[n],   g_t = a_t dh_t,   w_t = g_t h_{t-1},   dh0 = g_0,
//   du = delta sum_n dh B + skip v,   ddelta = u sum_n dh B + sum_n A w,
//   ddt = ddelta / (1 + exp(-dt - dt_bias)),   dz = dy y0 d/dz (z / (1 + exp(-z))),
//   dA = sum_{b,t} delta w,  dB_t = sum_d delta u dh,  dC_t = sum_d v h_t,
//   dskip = sum_{b,t} v u,   ddt_bias = sum_{b,t} ddt        (y0: y before the gate),
// and the single-token step.  States and all sums are float32.
//
// A block of four warps takes 128 / L channels of a stretch of tokens, L lanes a channel, four
// states a lane (L = N / 4, up to a power of two).  In tiles of sixteen tokens the threads
// form delta, delta u and v once for each token and channel and leave them in shared memory
// with B and C; then each lane walks its four states through the tile.  Sums over the
// states meet by shuffles, four tokens at a time, so that a lane ends with one
// finished sum; sums over channels (dB, dC) likewise, then over the warps in shared memory.
//
// Few channels: the tokens are cut into S segments that run side by side.  What a
// segment does to the state before it is h -> exp(A sum delta) h + H, H its result from a zero
// state; a first kernel forms H and sum delta of every segment, a second carries
// the states from segment to segment, and the third scans (likewise in reverse time).
// The forward leaves the state before every sixteenth token (a mark), from which the
// backward forms the states of a tile again.
//
// All sums are taken in a fixed order (parts of blocks are added by a last kernel): the same
// call gives the same bits.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "f32x2.cuh"
#include "pdl.cuh"
#include "sanatan_internal.h"
#include "sanatan_math.cuh"

namespace sanatan {
namespace {

using namespace f2;

constexpr int kTile = kSelectiveMark;  // tokens of a tile, and between two marks
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStates = 4;             // of a lane
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int L>
struct Geo {
  static constexpr int CW = 32 / L;          // channels of a warp
  static constexpr int CB = CW * kWarps;     // of a block
  static constexpr int NP = kStates * L;     // states, with those that fill up
  static constexpr int kCells = kTile * CB;  // (token, channel) pairs of a tile
  static constexpr int kItems = (kCells + kThreads - 1) / kThreads;  // of a thread
  static constexpr int kPairs = kTile * 2 * NP;   // values of B and C of a tile
  static constexpr int kPairItems = kPairs / kThreads;
  static constexpr int kPitch = CB + 8;  // (four tokens of eight channels: 32 banks)
};

__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum2(uint64_t v) {
  float a, b;
  upk2(v, a, b);
  return a + b;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^x of a pair.  The hardware's power of two is 0.3 steps of 2^-24 low next to 1, and a
// memory of n tokens multiplies the mean error of its decays by n; the first four terms of
// the series are within 0.15 steps for |x| < 1/32 (x ln 2 < 0.0217; the next is its fourth
// power / 24) and have no bias beside the rounding.  Beyond, memories are below 50 tokens.
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) {
  const uint64_t c1 = pk2(kLn2, kLn2), one = pk2(1.0f, 1.0f);
  const uint64_t c2 = pk2(0.24022650695910072f, 0.24022650695910072f);    // ln(2)^2 / 2
  const uint64_t c3 = pk2(0.055504108664821580f, 0.055504108664821580f);  // ln(2)^3 / 6
  const uint64_t p = ffma2(ffma2(ffma2(c3, x, c2), x, c1), x, one);
  float x0, x1, p0, p1;
  upk2(x, x0, x1);
  upk2(p, p0, p1);
  return pk2(fabsf(x0) < 0.03125f ? p0 : ex2(x0), fabsf(x1) < 0.03125f ? p1 : ex2(x1));
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// log(1 + exp(x)); for large x that is x.
__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.0f) + log1pf(__expf(-fabsf(x)));
}

__device__ __forceinline__ int length_of(const int64_t* lens, int b, int T) {
  if (lens == nullptr) return T;
  const int64_t n = lens[b];
  return n < 0 ? 0 : (n > T ? T : static_cast<int>(n));
}

// Halves M values a lane over lane bits LO .. HI (powers of two) while there are several, then
// sums over the bits left: lane ends with M / 2^k values, those from index() on.
template <int M, int LO, int HI>
struct Meet {
  static constexpr int halvings() {
    int n = M, bit = LO, k = 0;
    while (n > 1 && bit <= HI) n /= 2, bit *= 2, ++k;
    return k;
  }
  static constexpr int kLeft = M >> halvings();       // values of a lane at the end
  static constexpr int kDone = LO << halvings();      // the first bit not halved over
  __device__ __forceinline__ static void sum(float (&v)[M], int lane) {
    int bit = LO;
#pragma unroll
    for (int n = M / 2; n >= kLeft; n /= 2, bit *= 2) {
      if (n == 0) break;
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
      }
    }
    if constexpr (kDone <= HI)
#pragma unroll
      for (bit = kDone; bit <= HI; bit *= 2)
#pragma unroll
        for (int i = 0; i < kLeft; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], bit);
  }
  __device__ __forceinline__ static int index(int lane) {
    int k = 0, n = M / 2;
#pragma unroll
    for (int bit = LO; bit < kDone; bit *= 2, n /= 2) k += (lane & bit) ? n : 0;
    return k;
  }
  // Of the lanes that end with the same sum, the first.
  __device__ __forceinline__ static bool first(int lane) {
    return kDone > HI || (lane & (2 * HI - 1) & ~(kDone - 1)) == 0;
  }
};

// Where a block works.
template <int L>
struct Place {
  int b, seg, cb, tiles, k0, k1, n;  // k0 .. k1: the segment's tiles; n: tokens that are there
  __device__ __forceinline__ Place(const SelectiveArgs& a) {
    cb = blockIdx.x % a.blocks;
    const unsigned rest = blockIdx.x / a.blocks;
    seg = rest % a.segments;
    b = rest / a.segments;
    tiles = (a.T + kTile - 1) / kTile;
    k0 = seg * a.tiles_per_segment;
    k1 = min(k0 + a.tiles_per_segment, tiles);
    n = 0;
  }
};

// Four states of a lane in memory, [.., D, N].
struct StatePlace {
  int64_t at;   // of the lane's first state in a [D, N] slab
  int count;    // states of the lane that exist
  bool vec;
  __device__ __forceinline__ StatePlace(int d, int l, int D, int N, bool aligned) {
    at = static_cast<int64_t>(d) * N + kStates * l;
    count = d < D ? max(0, min(kStates, N - kStates * l)) : 0;
    vec = aligned && count == kStates;
  }
  __device__ __forceinline__ void load(const float* slab, float (&f)[kStates]) const {
    if (vec) {
      const float4 v = *reinterpret_cast<const float4*>(slab + at);
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < kStates; ++j) f[j] = j < count ? slab[at + j] : 0.0f;
    }
  }
  __device__ __forceinline__ void store(float* slab, uint64_t lo, uint64_t hi) const {
    float f[kStates];
    upk2(lo, f[0], f[1]);
    upk2(hi, f[2], f[3]);
    if (vec) {
      *reinterpret_cast<float4*>(slab + at) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
      for (int j = 0; j < kStates; ++j)
        if (j < count) slab[at + j] = f[j];
    }
  }
};

// B and C of a tile, loaded into registers, then put into shared memory [token][B | C][NP].
template <typename E, int L>
struct PairTile {
  using G = Geo<L>;
  float r[G::kPairItems];
  __device__ __forceinline__ void load(const SelectiveArgs& a, int b, int t0, int n) {
#pragma unroll
    for (int i = 0; i < G::kPairItems; ++i) {
      const int k = threadIdx.x + i * kThreads, s = k % G::NP, which = k / G::NP % 2;
      const int t = t0 + k / (2 * G::NP);
      const int64_t row = static_cast<int64_t>(b) * a.T + t;
      r[i] = 0.0f;
      if (t < n && s < a.N)
        r[i] = which == 0 ? load_as_float(static_cast<const E*>(a.Bm) + row * a.ldb + s)
                          : load_as_float(static_cast<const E*>(a.Cm) + row * a.ldc + s);
    }
  }
  __device__ __forceinline__ void put(float* pairs) const {
#pragma unroll
    for (int i = 0; i < G::kPairItems; ++i) pairs[threadIdx.x + i * kThreads] = r[i];
  }
};

// The carries of S segments, in place: H[b][s][D][N] becomes the state before segment s
// (reverse: the gradient behind it); sums [b][s][D] of delta.
__global__ void __launch_bounds__(256)
    selective_carry_kernel(float* H, const float* sums, const float* A, const float* first, int S,
                           int D, int N, int64_t all, bool reverse) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  wait_for_previous();
  if (i >= all) return;
  const int64_t slab = static_cast<int64_t>(D) * N, b = i / slab, at = i % slab, d = at / N;
  const float a = A[at] * kLog2e;
  float h = first != nullptr ? first[i] : 0.0f;
  for (int k = 0; k < S; ++k) {
    const int64_t s = b * S + (reverse ? S - 1 - k : k);
    const float own = H[s * slab + at], decay = ex2(a * sums[s * D + d]);
    H[s * slab + at] = h;
    h = fmaf(decay, h, own);
  }
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int64_t blocks, int threads, size_t shared,
                   cudaStream_t st, Args... args) {
  if (shared > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(shared));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_carry(const SelectiveArgs& a, const float* first, bool reverse,
                         cudaStream_t st) {
  const int64_t all = static_cast<int64_t>(a.B) * a.D * a.N;
  return launch(selective_carry_kernel, (all - 1) / 256 + 1, 256, 0, st, a.carry,
                static_cast<const float*>(a.sums), a.A, first, a.segments, a.D, a.N, all, reverse);
}

inline bool state_words(int N, std::initializer_list<const void*> states) {
  if (N % kStates != 0) return false;
  for (const void* p : states)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
  return true;
}

// f<E, L> for the lanes of a channel (a: the forward's arguments, in scope).
#define SANATAN_SELECTIVE_DISPATCH(f, E, args) \
  switch (selective_lanes(a.N)) {              \
    case 1:                                    \
      return f<E, 1>(args, st);                \
    case 2:                                    \
      return f<E, 2>(args, st);                \
    case 4:                                    \
      return f<E, 4>(args, st);                \
    case 8:                                    \
      return f<E, 8>(args, st);                \
    case 16:                                   \
      return f<E, 16>(args, st);               \
    default:                                   \
      return f<E, 32>(args, st);               \
  }

}  // namespace
}  // namespace sanatan
