// Gated linear recurrence, per channel of [B, T, D]:
//   h_t = a_t h_{t-1} + u_t,  y_t = h_t,
//   log gate:      a = exp(g),          u = x,
//   sigmoid gate:  a = 1/(1 + exp(-g)), u = (1 - a) x,
// its gradients
//   dh_t = dy_t + a_{t+1} dh_{t+1},  dh_{T-1} += dh_out,  dh0 = a_0 dh_0,
//   log gate:      dx = dh,          dg = dh a h_{t-1},
//   sigmoid gate:  dx = dh (1 - a),  dg = dh (h_{t-1} - x) a (1 - a),
// and the single-token step.  States and all sums are float32.
//
// A stretch of tokens is the affine map h -> A h + H of the state before it (A the
// product of its decays, H its result from a zero state), and maps compose: (A1, H1)
// then (A2, H2) is (A1 A2, A2 H1 + H2).  So every tensor is read once: a cluster of
// CTAs walks the tokens of 64 (or 32) channels of a sequence; in every step each CTA
// takes the next tile of 8192 (f32, backward: 4096) elements, 16 (8) lanes a run of
// eight (four) tokens of it, a lane four channels; the maps meet in registers, shared
// memory and, across the cluster, distributed shared memory, always in the same
// order (the same call gives the same bits), and the run's tokens follow from the state
// before it.  Tiles of the next two steps are under way meanwhile (TMA boxes).
// Arithmetic is packed, two channels an instruction.
//
// Bound: bytes (three tensors forward, five backward), and beside them the latency of
// a step: map, exchange, tokens.  Hence two CTAs an SM, and few steps rather than many
// warps.  Forward, training shape (B 8 T 4096 D 768, bf16, log gate), GB300: 28 us;
// half the run and three or four CTAs an SM 34 and 37 us, a third stage 29.4; as
// first built, a cluster barrier instead of st.async with a counting mbarrier made
// 44 us into 60 (the barrier's release waits for every thread's global stores), cp.async
// instead of TMA 27 into 32.  Device times of the measured copy rate: this forward
// 5.4 TB/s (0.80), its backward 48 us, 5.2 TB/s (0.77), with the sigmoid 29 and 55 us;
// B 1 T 32768 D 768, sigmoid, forward 37 us, 4.1 TB/s (0.60: one sequence's clusters do
// not fill the SMs evenly), backward 76 us, 3.3 TB/s (0.49: twice the steps).
// The same work without exchanges (24 sequences of 1408 tokens) takes 26.4 and 43.4 us.
//
// The backward needs h_{t-1}: the forward leaves the state before every 64th
// token (a mark, 1/64 of the elements in float32), from which a tile's states are
// recomputed with the same maps; reading y instead would cost as many bytes and
// its rounding.  In reverse time the map of a tile on the gradient that comes
// from later tokens is (A, P) with the same A.
#pragma once

#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "f32x2.cuh"
#include "pdl.cuh"
#include "per_device.h"
#include "sanatan_internal.h"
#include "sanatan_math.cuh"
#include "tc_ptx.cuh"

namespace sanatan {
namespace {

namespace cg = cooperative_groups;
using namespace f2;

constexpr int kMark = kScanMark;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kIssuer = kThreads - 32;  // the thread that issues the copies
constexpr int kMaxCluster = 16;
template <typename E>
constexpr int kRunFwd = sizeof(E) == 2 ? 8 : 4;  // consecutive tokens of a thread
constexpr int kRunBwd = 4;
constexpr int kStages = 2;  // tiles of a ring

// Four channels as two packed pairs.
struct V4 {
  uint64_t lo, hi;
};
__device__ __forceinline__ V4 v4(float a, float b, float c, float d) {
  return {pk2(a, b), pk2(c, d)};
}
__device__ __forceinline__ V4 v4(float a) { return v4(a, a, a, a); }
__device__ __forceinline__ V4 mul(const V4& a, const V4& b) {
  return {fmul2(a.lo, b.lo), fmul2(a.hi, b.hi)};
}
__device__ __forceinline__ V4 fma(const V4& a, const V4& b, const V4& c) {
  return {ffma2(a.lo, b.lo, c.lo), ffma2(a.hi, b.hi, c.hi)};
}
__device__ __forceinline__ V4 sub(const V4& a, const V4& b) {
  return {fsub2(a.lo, b.lo), fsub2(a.hi, b.hi)};
}
__device__ __forceinline__ V4 select(bool first, const V4& a, const V4& b) {
  return {first ? a.lo : b.lo, first ? a.hi : b.hi};
}
__device__ __forceinline__ void get(const V4& v, float (&f)[4]) {
  upk2(v.lo, f[0], f[1]);
  upk2(v.hi, f[2], f[3]);
}
__device__ __forceinline__ V4 shfl_xor(const V4& v, int mask) {
  float f[4];
  get(v, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = __shfl_xor_sync(0xffffffffu, f[j], mask);
  return v4(f[0], f[1], f[2], f[3]);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// The smaller of x and `most`; NaN stays NaN.
__device__ __forceinline__ float at_most(float x, float most) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(most));
  return r;
}

// a and 1 - a of four gate values.  A memory of n tokens multiplies the mean error of
// the decays by n, so decays next to 1 need more than the hardware's power of two,
// which is 0.3 steps of 2^-24 low there.  Log gate: exp(g) is the sum of its first five
// terms while |g| < 1/16 (the next is g^5 / 120, 0.13 steps at 1/16), the power of two
// beyond, where the rounded argument costs |g| steps of a small decay.  Sigmoid: with
// e = exp(-g) the sides are 1 / (1 + e) and e / (1 + e), so that each has its own digits
// where the other is next to 1.  The reciprocal r of the rounded 1 + e (its steps are
// 2^-23) is up to 1.9 steps off and 0.15 low on average for g in 2.8 ... 10; one step of
// Newton's iteration from the unrounded sum, r - r ((r - 1) + r e), rounds 1 / (1 + e)
// once (r.m.s. error 0.29 steps, mean 0.000).  Gates constant in time at 7 ... 10 over
// 32768 tokens: float32 output off by 3.8e-4 of itself (half a step of the decay over
// 1 - a is 6.6e-4 at 10), not 7.8e-4; long prefill 35.4 -> 37.1 us.  e stops at 2^126, so that
// neither side is 0 times infinity: decays are at least 2^-126.
template <int G>
__device__ __forceinline__ void gate(const V4& g, V4& a, V4& keep) {
  float t[4];
  if (G == SANATAN_GATE_LOG) {
    const V4 one = v4(1.0f);
    V4 sum = fma(g, v4(1.0f / 24), v4(1.0f / 6));
    sum = fma(sum, g, v4(0.5f));
    sum = fma(sum, g, one);
    sum = fma(sum, g, one);
    float near[4], f[4];
    get(mul(g, v4(kLog2e)), t);
    get(sum, near);
    get(g, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = fabsf(f[j]) < 0.0625f ? near[j] : ex2(t[j]);
    a = v4(t[0], t[1], t[2], t[3]);
  } else {
    get(mul(g, v4(-kLog2e)), t);
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = ex2(at_most(t[j], 126.0f));
    const V4 e = v4(t[0], t[1], t[2], t[3]), one = v4(1.0f);
    float s[4];
    get(fma(e, one, one), s);
    a = v4(rcp(s[0]), rcp(s[1]), rcp(s[2]), rcp(s[3]));
    keep = mul(e, a);
    a = sub(a, mul(a, fma(a, e, sub(a, one))));  // r - 1 is exact where it matters, r >= 1/2
  }
}

__device__ __forceinline__ int length_of(const int64_t* lens, int b, int T) {
  if (lens == nullptr) return T;
  const int64_t n = lens[b];
  return n < 0 ? 0 : (n > T ? T : static_cast<int>(n));
}

// Four values of a row in memory.
template <typename E>
struct Quad;
template <>
struct Quad<float> {
  using type = ulonglong2;
  __device__ __forceinline__ static V4 get(const ulonglong2& v) { return {v.x, v.y}; }
  __device__ __forceinline__ static ulonglong2 put(const V4& v) {
    return make_ulonglong2(v.lo, v.hi);
  }
};
template <>
struct Quad<__nv_bfloat16> {
  using type = uint2;
  __device__ __forceinline__ static V4 get(const uint2& v) {
    return v4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
              __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
  __device__ __forceinline__ static uint2 put(const V4& v) {
    float f[4];
    sanatan::get(v, f);
    const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(f[2], f[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                      *reinterpret_cast<const uint32_t*>(&hi));
  }
};

// A thread's four channels of the CTA's 4 * LANES.  TMA (D a multiple of 4): four
// neighbours, one load or store a row.  Otherwise rows start at any element:
// channels LANES apart, so that the lanes of a load are neighbours.
template <int LANES, bool TMA>
struct Place {
  int c0, lane, D;
  __device__ __forceinline__ int channel(int j) const {
    return TMA ? c0 + 4 * lane + j : c0 + lane + LANES * j;
  }
  __device__ __forceinline__ bool there(int j) const { return channel(j) < D; }
  template <typename E>
  __device__ __forceinline__ void store(E* row, const V4& v) const {
    if (TMA) {
      if (there(0)) *reinterpret_cast<typename Quad<E>::type*>(row + channel(0)) = Quad<E>::put(v);
    } else {
      float f[4];
      get(v, f);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (there(j)) row[channel(j)] = store_from_float<E>(f[j]);
    }
  }
};

// The same channels in pairs, pair < 2 * LANES, for the lanes of warp 0 (with 8
// LANES its upper half does what the lower one does).
template <int LANES, bool TMA>
struct PairPlace {
  int c[2];
  bool ok[2];
  __device__ __forceinline__ PairPlace(int c0, int pair, int D) {
    const Place<LANES, TMA> p{c0, pair / 2, D};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = p.channel(pair % 2 * 2 + i);
      ok[i] = c[i] < D;
    }
  }
  __device__ __forceinline__ uint64_t load(const float* row) const {  // zeros for null
    return pk2(row != nullptr && ok[0] ? row[c[0]] : 0.0f,
               row != nullptr && ok[1] ? row[c[1]] : 0.0f);
  }
  __device__ __forceinline__ void store(float* row, uint64_t v) const {
    float a, b;
    upk2(v, a, b);
    if (ok[0]) row[c[0]] = a;
    if (ok[1]) row[c[1]] = b;
  }
};

struct Maps {
  CUtensorMap of[3];
};

__device__ int g_scan_error;  // a bounded wait gave up

// The tensors' tiles on their way.  TMA (rows of a multiple of 16 bytes): a ring
// of STAGES tiles in shared memory, each tensor's tile one box copy that one
// thread issues (rows past T and channels past D come as zeros).  Otherwise the
// next tile waits in registers.
template <typename E, int LANES, bool TMA, int NT, int R, int STAGES>
struct Tiles {
  static constexpr int kTile = kThreads / LANES * R;
  static constexpr int kWidth = 4 * LANES;
  static constexpr int kBox = kTile * kWidth * static_cast<int>(sizeof(E));
  static constexpr int kBytes = TMA ? STAGES * NT * kBox : 0;
  using Q = typename Quad<E>::type;
  const E* src[NT];  // registers: the thread's first channel of token 0
  int64_t D;
  int b, len;
  Place<LANES, TMA> place;
  unsigned char* ring;
  uint64_t* full;    // [STAGES] mbarriers
  const unsigned char* own;  // the thread's first values of a tile
  const Maps* maps;
  bool* dead;
  E next[TMA ? 1 : NT][TMA ? 1 : R][4];

  __device__ __forceinline__ void start(int tid) {
    if constexpr (TMA) {
      own = ring + (tid / LANES * R * kWidth + 4 * (tid % LANES)) * static_cast<int>(sizeof(E));
      if (tid == 0)
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(&full[i], 1);
      tc::fence_mbar_init();
      if (tid == kIssuer)
#pragma unroll
        for (int i = 0; i < NT; ++i)
          asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps->of[i]))
                       : "memory");
    }
  }
  // TMA, one thread: fetch the tile that starts at token t (none of it present:
  // only complete the phase).
  __device__ __forceinline__ void fetch(int t, int slot) {
    if (t >= len) {
      tc::mbar_arrive(&full[slot]);
      return;
    }
    tc::mbar_arrive_expect_tx(&full[slot], NT * kBox);
#pragma unroll
    for (int i = 0; i < NT; ++i)
      asm volatile(
          "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
          " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tc::smem_u32(ring + (slot * NT + i) * kBox)),
          "l"(reinterpret_cast<uint64_t>(&maps->of[i])), "r"(place.c0), "r"(t), "r"(b),
          "r"(tc::smem_u32(&full[slot]))
          : "memory");
  }
  __device__ __forceinline__ void wait(int slot, uint32_t parity) {
    if (!*dead && !tc::mbar_wait_bounded(&full[slot], parity)) {
      *dead = true;
      g_scan_error = 1;
    }
  }
  // Registers: the thread's tokens t0 ... of a tile.
  __device__ __forceinline__ void prefetch(int t0) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          next[i][r][j] = t0 + r < len && place.there(j)
                              ? src[i][(static_cast<int64_t>(t0) + r) * D + LANES * j]
                              : store_from_float<E>(0.0f);
  }
  __device__ __forceinline__ V4 get(int i, int r, int slot) const {
    if constexpr (TMA)
      return Quad<E>::get(*reinterpret_cast<const Q*>(
          own + (slot * NT + i) * kBox + r * kWidth * static_cast<int>(sizeof(E))));
    else
      return v4(load_as_float(&next[i][r][0]), load_as_float(&next[i][r][1]),
                load_as_float(&next[i][r][2]), load_as_float(&next[i][r][3]));
  }
};

__device__ __forceinline__ uint64_t* pairs(V4* v) { return &v->lo; }

// One step's exchange.  Channel pairs: lane l of a run has the pairs 2 l and 2 l + 1
// (V4 rows read as pairs).
template <int LANES, bool BWD>
struct Exchange {
  V4 a[kWarps][LANES];   // the maps of the CTA's warps
  V4 h[kWarps][LANES];
  V4 in[kWarps][LANES];  // what comes into each warp
  V4 p[BWD ? kWarps : 1][LANES];  // the same in reverse time
  V4 in_p[BWD ? kWarps : 1][LANES];
  uint64_t full[2];      // mbarriers: all of a step's maps have come
  uint64_t ring[kStages];  // mbarriers: a tile has come
};

// Phase `bar` completes once `bytes` have come.  Relaxed: nothing the thread did
// before has to be seen by anyone (a release would wait for its global stores).
__device__ __forceinline__ void expect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\t"
      "mbarrier.arrive.expect_tx.relaxed.cluster.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(
          tc::smem_u32(bar)),
      "r"(bytes)
      : "memory");
}

// The cluster's side of the recurrence, by warp 0, lane = channel pair.  A step:
// share() sends the CTA's map to every CTA of the cluster (st.async, counted by
// the receiver's mbarrier and acquired at cluster scope; a cluster barrier instead
// would make every thread wait for its own global stores), arrive() waits for all of
// them and takes carry over them.  Buffers alternate: who sends step s + 2 has received
// step s + 1 from every CTA, and they sent that after reading step s.
template <int LANES, bool BWD>
struct Cluster {
  Exchange<LANES, BWD>& ex;
  ulonglong2* all;  // [2][size][2 * LANES]: (A, H) of the cluster's CTAs, by the step's parity
  int rank, size, steps, pair;
  bool dead = false;  // a wait gave up: no more waiting

  __device__ __forceinline__ ulonglong2* of(int s, int r) const {
    return all + ((s & 1) * size + r) * 2 * LANES + pair;
  }
  __device__ __forceinline__ uint32_t bytes() const { return size * 2 * LANES * 16; }
  __device__ __forceinline__ void start() {  // all threads
    if (size == 1) {
      __syncthreads();
      return;
    }
    if (threadIdx.x == 0) {
      tc::mbar_init(&ex.full[0], 1);
      tc::mbar_init(&ex.full[1], 1);
      tc::fence_mbar_init();
      expect(&ex.full[0], bytes());
      expect(&ex.full[1], bytes());
    }
    cg::this_cluster().sync();
  }
  __device__ __forceinline__ void share(int s, uint64_t A, uint64_t H) {
    if (threadIdx.x >= 2 * LANES) return;
    const uint32_t at = tc::smem_u32(of(s, rank)), bar = tc::smem_u32(&ex.full[s & 1]);
    for (int r = 0; r < size; ++r) {
      uint32_t to, to_bar;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(r));
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to_bar) : "r"(bar), "r"(r));
      asm volatile(
          "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64"
          " [%0], {%1, %2}, [%3];" ::"r"(to),
          "l"(A), "l"(H), "r"(to_bar)
          : "memory");
    }
  }
  // What comes into this CTA's tile of step s.
  __device__ __forceinline__ uint64_t arrive(int s, uint64_t& carry) {
    if (!dead && !tc::mbar_wait_cluster_bounded(&ex.full[s & 1], (s >> 1) & 1)) {
      dead = true;
      g_scan_error = 1;
    }
    uint64_t in = carry;
    for (int r = 0; r < size; ++r) {
      const ulonglong2 m = *of(s, r);
      if (r == rank) in = carry;
      carry = ffma2(m.x, carry, m.y);
    }
    __syncwarp();
    if (threadIdx.x == 0 && s + 2 < steps) expect(&ex.full[s & 1], bytes());
    return in;
  }
  // No CTA leaves while another may still send to it, or its own copies are under way.
  __device__ __forceinline__ void finish() {
    if (dead) __nanosleep(1000000);  // copies under way land
    if (size == 1) return;
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    asm volatile("barrier.cluster.wait;" ::: "memory");
  }
};

// The maps of the 32 / LANES runs of a warp: (wA, wH) all of them in order, (bA,
// bH) those before the thread's own.  Forward in time, or backward.
template <int LANES, bool REVERSE>
__device__ __forceinline__ void warp_scan(int tid, const V4& A, const V4& H, V4& bA, V4& bH, V4& wA,
                                          V4& wH) {
  bA = v4(1.0f);
  bH = v4(0.0f);
  wA = A;
  wH = H;
#pragma unroll
  for (int off = LANES; off < 32; off *= 2) {
    const V4 oA = shfl_xor(wA, off), oH = shfl_xor(wH, off);
    const bool second = ((tid & off) != 0) != REVERSE;  // the other half comes before
    const V4 nH = second ? fma(wA, oH, wH) : fma(oA, wH, oH);
    if (second) {
      bH = fma(bA, oH, bH);
      bA = mul(bA, oA);
    }
    wH = nH;
    wA = mul(wA, oA);
  }
}

constexpr int exchange_bytes(int cluster, int lanes) { return 2 * cluster * 2 * lanes * 16; }

// cuTensorMapEncodeTiled, looked up through the runtime until it is found.
PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PerDevice<PFN_cuTensorMapEncodeTiled_v12000, 1> known;
  PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  const cudaError_t e = known.get(0, &fn, [](PFN_cuTensorMapEncodeTiled_v12000* out) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                           cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess) return cudaErrorSymbolNotFound;
    *out = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    return cudaSuccess;
  });
  if (e == cudaSuccess) return fn;
  cudaGetLastError();  // (the call goes on without tensor maps)
  return nullptr;
}

// The map of a [B, T, D] tensor (rows of a multiple of 16 bytes) with boxes of `rows`
// tokens x `width` channels; false where none can be made (sizes out of the
// format's range).
bool encode(CUtensorMap* map, const void* p, int dtype, int B, int T, int D, int rows, int width) {
  const cuuint64_t e = dtype == SANATAN_F32 ? 4 : 2;
  const PFN_cuTensorMapEncodeTiled_v12000 encoder = map_encoder();
  if (encoder == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(T),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[2] = {D * e, static_cast<cuuint64_t>(T) * D * e};
  if (strides[1] >= (1ull << 40)) return false;
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return encoder(map,
                 dtype == SANATAN_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                 3, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch shape: CTAs of a cluster, and the steps that the longest CTA takes (over
// all waves of clusters).
struct Shape {
  int cluster;
  int64_t steps;
};

template <typename Args, typename Ring>
cudaLaunchConfig_t config(int64_t ctas, int cluster, cudaLaunchAttribute* attr, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Ring::kBytes + exchange_bytes(cluster, Ring::kWidth / 4);
  cfg.stream = st;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = cluster;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// held[n]: clusters of n CTAs of a kernel that the current device holds at once.  The
// runtime is asked once a device (again after a failure), when the kernel's attributes are
// set too.
struct Held {
  int held[kMaxCluster + 1] = {};
};
template <auto Kernel, typename Args, typename Ring>
cudaError_t ask(Held* out) {
  const void* fn = reinterpret_cast<const void*>(Kernel);
  cudaError_t e =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Ring::kBytes + exchange_bytes(kMaxCluster, Ring::kWidth / 4));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int n = 1; e == cudaSuccess && n <= kMaxCluster; ++n) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config<Args, Ring>(n, n, attr, nullptr);
    e = cudaOccupancyMaxActiveClusters(&out->held[n], Kernel, &cfg);
    if (e == cudaErrorInvalidClusterSize || e == cudaErrorInvalidConfiguration ||
        e == cudaErrorLaunchOutOfResources) {  // none of this size
      cudaGetLastError();
      out->held[n] = 0;
      e = cudaSuccess;
    }
  }
  return e;
}
template <auto Kernel, typename Args, typename Ring>
cudaError_t held_by(Held* out) {
  static PerDevice<Held> known;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : known.get(dev, out, ask<Kernel, Args, Ring>);
}

// Few sequences: the largest cluster with which all clusters still run at once (a
// second wave would cost more than it splits), and of those with the same
// number of steps the smallest.  Training shape (B 8, T 4096, D 768, bf16: 96
// blocks of 64 channels), forward and backward us by cluster size: 1: 35 and 73, 2: 35
// and 63, 3: 28 and 49 (288 of 291 places), 4: 32 and 58, 8: 36 and 58.
template <auto Kernel, typename Args, typename Ring>
cudaError_t shape_of(const Args& a, Shape* best) {
  Held h;
  const cudaError_t e = held_by<Kernel, Args, Ring>(&h);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.B) * ((a.D + Ring::kWidth - 1) / Ring::kWidth);
  const int64_t tiles = (static_cast<int64_t>(a.T) + Ring::kTile - 1) / Ring::kTile;
  *best = {1, tiles * (h.held[1] > 0 ? (units + h.held[1] - 1) / h.held[1] : units)};
  for (int n = 2; n <= kMaxCluster && n <= tiles; ++n) {
    const int64_t steps = (tiles + n - 1) / n;
    if (units <= h.held[n] && steps < best->steps) *best = {n, steps};
  }
  return cudaSuccess;
}

template <auto Kernel, typename Args, typename Ring>
cudaError_t launch(const Args& a, const Maps& maps, int cluster, cudaStream_t st) {
  const int blocks = (a.D + Ring::kWidth - 1) / Ring::kWidth;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      config<Args, Ring>(static_cast<int64_t>(a.B) * blocks * cluster, cluster, attr, st);
  return cudaLaunchKernelEx(&cfg, Kernel, a, maps, blocks, cluster);
}

// Channels of a CTA: 64 or 32, whichever takes fewer steps (tiles of 32 channels have
// twice the tokens; they let few sequences fill the GPU).
template <auto Wide, auto Narrow, typename Args, typename WideRing, typename NarrowRing>
cudaError_t launch_best(const Args& a, bool (*encode_all)(Maps*, const Args&, int, int),
                        cudaStream_t st, bool* encoded) {
  Shape w, n;
  cudaError_t e = shape_of<Wide, Args, WideRing>(a, &w);
  if (e == cudaSuccess) e = shape_of<Narrow, Args, NarrowRing>(a, &n);
  if (e != cudaSuccess) {
    *encoded = true;
    return e;
  }
  Maps m;
  if (n.steps < w.steps) {
    *encoded = encode_all(&m, a, NarrowRing::kTile, NarrowRing::kWidth);
    return *encoded ? launch<Narrow, Args, NarrowRing>(a, m, n.cluster, st) : cudaSuccess;
  }
  *encoded = encode_all(&m, a, WideRing::kTile, WideRing::kWidth);
  return *encoded ? launch<Wide, Args, WideRing>(a, m, w.cluster, st) : cudaSuccess;
}

template <typename Args>
bool encode_none(Maps*, const Args&, int, int) {
  return true;
}

// Whether a bounded wait of this translation unit's kernels gave up since the last
// call (1; cleared), or -1 for a CUDA error.
inline int read_and_clear_error(cudaStream_t st) {
  int h = 0;
  if (cudaMemcpyFromSymbolAsync(&h, g_scan_error, sizeof(int), 0, cudaMemcpyDeviceToHost, st) !=
      cudaSuccess)
    return -1;
  if (cudaStreamSynchronize(st) != cudaSuccess) return -1;
  if (h != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_scan_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) !=
        cudaSuccess)
      return -1;
    if (cudaStreamSynchronize(st) != cudaSuccess) return -1;
  }
  return h;
}

}  // namespace
}  // namespace sanatan
