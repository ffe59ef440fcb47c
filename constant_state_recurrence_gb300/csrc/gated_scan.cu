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
// A stretch of tokens is the affine map h -> A h + H of the state before it
// (A the product of its decays, H its result from a zero state), and maps
// compose: (A1, H1) then (A2, H2) is (A1 A2, A2 H1 + H2).  So every tensor is
// read once: a cluster of CTAs walks the tokens of 64 channels of a sequence, in
// every step each CTA takes the next tile, each half-warp kRun consecutive tokens
// of it (a lane four channels), and the maps meet in registers, shared memory and,
// across the cluster, distributed shared memory, always in the same order (the
// same call gives the same bits).  One cluster barrier a step; tiles of later
// steps are on their way meanwhile (cp.async into a ring that each thread fills
// and reads for itself).
//
// The backward needs h_{t-1}: the forward leaves the state before every 64th
// token (a mark, 1/64 of the elements in float32), from which a tile's states are
// recomputed with the same maps; reading y instead would cost as many bytes and
// its rounding.  In reverse time the map of a tile on the gradient that comes
// from later tokens is (A, P) with the same A.
#include <cooperative_groups.h>

#include "sanatan_internal.h"
#include "sanatan_math.cuh"

namespace sanatan {
namespace {

namespace cg = cooperative_groups;

constexpr int kMark = kScanMark;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRuns = kThreads / 16;  // half-warps
constexpr int kChannels = 64;         // of a CTA: 16 lanes x 4
constexpr int kMaxCluster = 8;

// a and 1 - a of a gate value; the sigmoid's two sides come from exp(-|g|), so
// neither overflows nor loses digits next to 1.
template <int G>
__device__ __forceinline__ void gate(float g, float& a, float& keep) {
  if (G == SANATAN_GATE_LOG) {
    a = expf(g);
    keep = 1.0f;
  } else {
    const float e = expf(-fabsf(g));
    const float r = 1.0f / (1.0f + e);
    const float q = e * r;
    a = g >= 0.0f ? r : q;
    keep = g >= 0.0f ? q : r;
  }
}

__device__ __forceinline__ int length_of(const int64_t* lens, int b, int T) {
  if (lens == nullptr) return T;
  const int64_t n = lens[b];
  return n < 0 ? 0 : (n > T ? T : static_cast<int>(n));
}

template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void unpack(const float4& v, float (&f)[4]) {
  f[0] = v.x;
  f[1] = v.y;
  f[2] = v.z;
  f[3] = v.w;
}
__device__ __forceinline__ void unpack(const uint2& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xffff0000u);
}
template <typename E>
struct Quad;  // four values of a row
template <>
struct Quad<float> {
  using type = float4;
  __device__ static float4 pack(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Quad<__nv_bfloat16> {
  using type = uint2;
  __device__ static uint2 pack(const float (&f)[4]) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(f[2], f[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                      *reinterpret_cast<const uint32_t*>(&hi));
  }
};

// Where a thread's four channels are.  VEC (D a multiple of 4): four neighbours,
// one load or store a row.  Otherwise rows start at any element: channels 16
// apart, so that the 16 lanes of a load are neighbours.
template <bool VEC>
__device__ __forceinline__ int channel(int c0, int lane, int j) {
  return VEC ? c0 + 4 * lane + j : c0 + lane + 16 * j;
}

template <typename E, bool VEC>
__device__ __forceinline__ void store_row(E* row, int c0, int lane, int D, const float (&f)[4]) {
  if (VEC) {
    if (channel<VEC>(c0, lane, 0) < D)
      *reinterpret_cast<typename Quad<E>::type*>(row + channel<VEC>(c0, lane, 0)) =
          Quad<E>::pack(f);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (channel<VEC>(c0, lane, j) < D)
        row[channel<VEC>(c0, lane, j)] = store_from_float<E>(f[j]);
  }
}

__device__ __forceinline__ float4 f4(const float (&f)[4]) {
  return make_float4(f[0], f[1], f[2], f[3]);
}

// The tensors' tiles on their way.  VEC: a ring of kStages tiles in shared memory,
// in which every thread has its own places (no barrier).  Otherwise the next tile
// waits in registers.
template <typename E, bool VEC, int NT, int R, int STAGES>
struct Tiles {
  using Q = typename Quad<E>::type;
  static constexpr int kBytes = VEC ? STAGES * NT * R * kThreads * static_cast<int>(sizeof(Q)) : 0;
  const E* src[NT];
  int64_t base;  // element of token 0, channel of lane and j = 0
  int c0, lane, D, len, tid;
  uint32_t ring;
  Q* ring_ptr;
  E next[VEC ? 1 : NT][VEC ? 1 : R][4];

  // Loads of tile `k` of this thread (tokens t0 ...; those from len on are not there).
  __device__ __forceinline__ void issue(int t0, int slot) {
    if constexpr (VEC) {
      if (channel<VEC>(c0, lane, 0) < D) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (t0 + r < len)
              cp_async<sizeof(Q)>(
                  ring + static_cast<uint32_t>((((slot * NT + i) * R + r) * kThreads + tid) *
                                               static_cast<int>(sizeof(Q))),
                  src[i] + base + static_cast<int64_t>(t0 + r) * D);
      }
      cp_commit();
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            next[i][r][j] = t0 + r < len && channel<VEC>(c0, lane, j) < D
                                ? src[i][base + static_cast<int64_t>(t0 + r) * D + 16 * j]
                                : store_from_float<E>(0.0f);
    }
  }
  __device__ __forceinline__ void get(int i, int r, int slot, float (&f)[4]) const {
    if constexpr (VEC) {
      unpack(ring_ptr[((slot * NT + i) * R + r) * kThreads + tid], f);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = load_as_float(&next[i][r][j]);
    }
  }
};

template <typename E>
constexpr int kRunFwd = sizeof(E) == 2 ? 8 : 4;  // tokens of a half-warp's run
constexpr int kStagesFwd = 3;

// One step's exchange: the maps of a CTA's tile, and of all tiles of the cluster.
struct Shared {
  float4 a[kWarps][16];
  float4 h[kWarps][16];
  float4 p[kWarps][16];
  float4 all_a[2][kMaxCluster][16];  // by parity of the step
  float4 all_h[2][kMaxCluster][16];
};

// then: the map (a, h) after the map (pa, ph).
__device__ __forceinline__ void then(float (&pa)[4], float (&ph)[4], const float4& a,
                                     const float4& h) {
  float fa[4], fh[4];
  unpack(a, fa);
  unpack(h, fh);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    ph[j] = fmaf(fa[j], ph[j], fh[j]);
    pa[j] *= fa[j];
  }
}

template <typename E, int G, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) scan_fwd_kernel(const ScanArgs p, int blocks,
                                                               int cluster_size) {
  constexpr int R = kRunFwd<E>;
  constexpr int kTile = kRuns * R;
  using Ring = Tiles<E, VEC, 2, R, kStagesFwd>;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();

  const int rank = static_cast<int>(blockIdx.x % cluster_size);
  const int unit = static_cast<int>(blockIdx.x / cluster_size);
  const int b = unit / blocks;
  const int tid = threadIdx.x, lane = tid & 15, warp = tid >> 5;
  const bool upper = (tid & 16) != 0;
  const int T = p.T, D = p.D;
  const int c0 = (unit % blocks) * kChannels;
  const int len = length_of(p.lens, b, T);
  const int run = (tid >> 4) * R;  // first token of this half-warp's run in a tile
  const int tiles = (T + kTile - 1) / kTile;
  const int steps = (tiles + cluster_size - 1) / cluster_size;

  Ring in;
  in.src[0] = static_cast<const E*>(p.g);
  in.src[1] = static_cast<const E*>(p.x);
  in.base = static_cast<int64_t>(b) * T * D + channel<VEC>(c0, lane, 0);
  in.c0 = c0;
  in.lane = lane;
  in.D = D;
  in.len = len;
  in.tid = tid;
  in.ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  in.ring_ptr = reinterpret_cast<typename Ring::Q*>(ring);
  E* y = static_cast<E*>(p.y) + static_cast<int64_t>(b) * T * D;
  const int marks_of = (T + kMark - 1) / kMark;

  float carry[4];  // the state before the step's first tile
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = channel<VEC>(c0, lane, j);
    carry[j] = p.h0 != nullptr && c < D ? p.h0[static_cast<int64_t>(b) * D + c] : 0.0f;
  }

  const int stride = cluster_size * kTile;
  const int64_t first = static_cast<int64_t>(rank) * kTile + run;
  // Token of step s; steps past the last one load nothing.
  auto token = [&](int s) {
    const int64_t t = first + static_cast<int64_t>(s) * stride;
    return t < T ? static_cast<int>(t) : T;
  };
  if constexpr (VEC) {
#pragma unroll
    for (int s = 0; s < kStagesFwd - 1; ++s) in.issue(token(s), s);
  } else {
    in.issue(token(0), 0);
  }

  int slot = 0;
  for (int s = 0; s < steps; ++s) {
    const int t0 = token(s);
    if constexpr (VEC) {
      in.issue(token(s + kStagesFwd - 1), slot == 0 ? kStagesFwd - 1 : slot - 1);
      cp_wait<kStagesFwd - 1>();
    }
    // The run's decays and inputs, and its map.
    float a[R][4], u[R][4], A[4] = {1.0f, 1.0f, 1.0f, 1.0f}, H[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float g[4], x[4];
      in.get(0, r, slot, g);
      in.get(1, r, slot, x);
      const bool there = t0 + r < len;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float keep;
        gate<G>(g[j], a[r][j], keep);
        u[r][j] = G == SANATAN_GATE_LOG ? x[j] : keep * x[j];
        if (!there) {
          a[r][j] = 1.0f;
          u[r][j] = 0.0f;
        }
        H[j] = fmaf(a[r][j], H[j], u[r][j]);
        A[j] *= a[r][j];
      }
    }
    if constexpr (!VEC) in.issue(token(s + 1), 0);
    // The two runs of the warp, then the warps of the CTA.
    float oA[4], oH[4], wA[4], wH[4];  // the other run's map; the warp's
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      oA[j] = __shfl_xor_sync(0xffffffffu, A[j], 16);
      oH[j] = __shfl_xor_sync(0xffffffffu, H[j], 16);
      wA[j] = A[j] * oA[j];
      wH[j] = upper ? fmaf(A[j], oH[j], H[j]) : fmaf(oA[j], H[j], oH[j]);
    }
    if (!upper) {
      sh.a[warp][lane] = f4(wA);
      sh.h[warp][lane] = f4(wH);
    }
    __syncthreads();
    float pA[4] = {1.0f, 1.0f, 1.0f, 1.0f}, pH[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = 0; w < warp; ++w) then(pA, pH, sh.a[w][lane], sh.h[w][lane]);
    if (warp == kWarps - 1) {  // the CTA's map, to every CTA of the cluster
      float tA[4], tH[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        tA[j] = pA[j] * wA[j];
        tH[j] = fmaf(wA[j], pH[j], wH[j]);
      }
      for (int r = upper ? 1 : 0; r < cluster_size; r += 2) {
        *cluster.map_shared_rank(&sh.all_a[s & 1][rank][lane], r) = f4(tA);
        *cluster.map_shared_rank(&sh.all_h[s & 1][rank][lane], r) = f4(tH);
      }
    }
    cluster.sync();
    // The state before this CTA's tile, and after the step's last.
    float h[4] = {carry[0], carry[1], carry[2], carry[3]};
    for (int r = 0; r < cluster_size; ++r) {
      float fa[4], fh[4];
      unpack(sh.all_a[s & 1][r][lane], fa);
      unpack(sh.all_h[s & 1][r][lane], fh);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r == rank) h[j] = carry[j];
        carry[j] = fmaf(fa[j], carry[j], fh[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = fmaf(pA[j], h[j], pH[j]);
      if (upper) h[j] = fmaf(oA[j], h[j], oH[j]);
    }
    if (p.marks != nullptr && t0 % kMark == 0 && t0 < T)
      store_row<float, VEC>(
          p.marks + (static_cast<int64_t>(b) * marks_of + t0 / kMark) * D, c0, lane, D, h);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float out[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = fmaf(a[r][j], h[j], u[r][j]);
        out[j] = t0 + r < len ? h[j] : 0.0f;
      }
      if (t0 + r < T) store_row<E, VEC>(y + static_cast<int64_t>(t0 + r) * D, c0, lane, D, out);
    }
    slot = slot == kStagesFwd - 1 ? 0 : slot + 1;
  }
  if (p.h_out != nullptr && rank == 0 && tid < 16)
    store_row<float, VEC>(p.h_out + static_cast<int64_t>(b) * D, c0, lane, D, carry);
}

constexpr int kRunBwd = kMark / kRuns;  // a tile lies between two marks
constexpr int kStagesBwd = 2;

template <typename E, int G, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(const ScanBwdArgs p, int blocks,
                                                               int cluster_size) {
  constexpr int R = kRunBwd;
  constexpr int kTile = kRuns * R;
  using Ring = Tiles<E, VEC, 3, R, kStagesBwd>;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();

  const int rank = static_cast<int>(blockIdx.x % cluster_size);
  const int unit = static_cast<int>(blockIdx.x / cluster_size);
  const int b = unit / blocks;
  const int tid = threadIdx.x, lane = tid & 15, warp = tid >> 5;
  const bool upper = (tid & 16) != 0;
  const int T = p.T, D = p.D;
  const int c0 = (unit % blocks) * kChannels;
  const int len = length_of(p.lens, b, T);
  const int run = (tid >> 4) * R;
  const int tiles = (T + kTile - 1) / kTile;
  const int steps = (tiles + cluster_size - 1) / cluster_size;

  Ring in;
  in.src[0] = static_cast<const E*>(p.g);
  in.src[1] = static_cast<const E*>(p.x);
  in.src[2] = static_cast<const E*>(p.dy);
  in.base = static_cast<int64_t>(b) * T * D + channel<VEC>(c0, lane, 0);
  in.c0 = c0;
  in.lane = lane;
  in.D = D;
  in.len = len;
  in.tid = tid;
  in.ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  in.ring_ptr = reinterpret_cast<typename Ring::Q*>(ring);
  E* dx = static_cast<E*>(p.dx) + static_cast<int64_t>(b) * T * D;
  E* dg = static_cast<E*>(p.dg) + static_cast<int64_t>(b) * T * D;

  float carry[4];  // gradient that comes into the step's last token from later ones
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = channel<VEC>(c0, lane, j);
    carry[j] = p.dh_out != nullptr && c < D ? p.dh_out[static_cast<int64_t>(b) * D + c] : 0.0f;
  }

  // Tile of step s: rank 0 has the last one, rank 1 the one before it, and so on;
  // -1 past the first.
  auto tile = [&](int s) {
    const int64_t k = tiles - 1 - (static_cast<int64_t>(s) * cluster_size + rank);
    return k < 0 ? -1 : static_cast<int>(k);
  };
  auto token = [&](int s) {
    const int k = tile(s);
    return k < 0 ? T : k * kTile + run;
  };
  if constexpr (VEC) {
#pragma unroll
    for (int s = 0; s < kStagesBwd - 1; ++s) in.issue(token(s), s);
  } else {
    in.issue(token(0), 0);
  }

  int slot = 0;
  for (int s = 0; s < steps; ++s) {
    const int k = tile(s);
    const int t0 = token(s);
    float h[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // the state before the tile
    if (k >= 0) {
      const float* mark = p.marks + (static_cast<int64_t>(b) * tiles + k) * D;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (channel<VEC>(c0, lane, j) < D) h[j] = mark[channel<VEC>(c0, lane, j)];
    }
    if constexpr (VEC) {
      in.issue(token(s + kStagesBwd - 1), slot == 0 ? kStagesBwd - 1 : slot - 1);
      cp_wait<kStagesBwd - 1>();
    }
    float a[R][4], keep[R][4], x[R][4], dy[R][4];
    float A[4] = {1.0f, 1.0f, 1.0f, 1.0f}, H[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float P[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float g[4];
      in.get(0, r, slot, g);
      in.get(1, r, slot, x[r]);
      in.get(2, r, slot, dy[r]);
      const bool there = t0 + r < len;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        gate<G>(g[j], a[r][j], keep[r][j]);
        if (!there) {
          a[r][j] = 1.0f;
          keep[r][j] = x[r][j] = dy[r][j] = 0.0f;
        }
        H[j] = fmaf(a[r][j], H[j], G == SANATAN_GATE_LOG ? x[r][j] : keep[r][j] * x[r][j]);
        A[j] *= a[r][j];
      }
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
#pragma unroll
      for (int j = 0; j < 4; ++j) P[j] = a[r][j] * (P[j] + dy[r][j]);
    if constexpr (!VEC) in.issue(token(s + 1), 0);
    float oA[4], oH[4], oP[4], wA[4], wH[4], wP[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      oA[j] = __shfl_xor_sync(0xffffffffu, A[j], 16);
      oH[j] = __shfl_xor_sync(0xffffffffu, H[j], 16);
      oP[j] = __shfl_xor_sync(0xffffffffu, P[j], 16);
      wA[j] = A[j] * oA[j];
      wH[j] = upper ? fmaf(A[j], oH[j], H[j]) : fmaf(oA[j], H[j], oH[j]);
      wP[j] = upper ? fmaf(oA[j], P[j], oP[j]) : fmaf(A[j], oP[j], P[j]);
    }
    if (!upper) {
      sh.a[warp][lane] = f4(wA);
      sh.h[warp][lane] = f4(wH);
      sh.p[warp][lane] = f4(wP);
    }
    __syncthreads();
    float pA[4] = {1.0f, 1.0f, 1.0f, 1.0f}, pP[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = 0; w < warp; ++w) {  // states: the warps before this one
      float fa[4], fh[4];
      unpack(sh.a[w][lane], fa);
      unpack(sh.h[w][lane], fh);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = fmaf(fa[j], h[j], fh[j]);
    }
    for (int w = kWarps - 1; w > warp; --w)  // gradients: the warps after it
      then(pA, pP, sh.a[w][lane], sh.p[w][lane]);
    if (warp == 0) {
      float tA[4], tP[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        tA[j] = pA[j] * wA[j];
        tP[j] = fmaf(wA[j], pP[j], wP[j]);
      }
      for (int r = upper ? 1 : 0; r < cluster_size; r += 2) {
        *cluster.map_shared_rank(&sh.all_a[s & 1][rank][lane], r) = f4(tA);
        *cluster.map_shared_rank(&sh.all_h[s & 1][rank][lane], r) = f4(tP);
      }
    }
    cluster.sync();
    float d[4] = {carry[0], carry[1], carry[2], carry[3]};
    for (int r = 0; r < cluster_size; ++r) {
      float fa[4], fp[4];
      unpack(sh.all_a[s & 1][r][lane], fa);
      unpack(sh.all_h[s & 1][r][lane], fp);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r == rank) d[j] = carry[j];
        carry[j] = fmaf(fa[j], carry[j], fp[j]);
      }
    }
    float before[R][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[j] = fmaf(pA[j], d[j], pP[j]);
      if (!upper) d[j] = fmaf(oA[j], d[j], oP[j]);
      if (upper) h[j] = fmaf(oA[j], h[j], oH[j]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        before[r][j] = h[j];
        h[j] = fmaf(a[r][j], h[j], G == SANATAN_GATE_LOG ? x[r][j] : keep[r][j] * x[r][j]);
      }
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float ox[4], og[4];
      const bool there = t0 + r < len;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float dh = dy[r][j] + d[j];
        d[j] = a[r][j] * dh;
        if (G == SANATAN_GATE_LOG) {
          ox[j] = dh;
          og[j] = d[j] * before[r][j];
        } else {
          ox[j] = dh * keep[r][j];
          og[j] = dh * ((before[r][j] - x[r][j]) * (a[r][j] * keep[r][j]));
        }
        if (!there) ox[j] = og[j] = 0.0f;
      }
      if (t0 + r < T) {
        store_row<E, VEC>(dx + static_cast<int64_t>(t0 + r) * D, c0, lane, D, ox);
        store_row<E, VEC>(dg + static_cast<int64_t>(t0 + r) * D, c0, lane, D, og);
      }
    }
    slot = slot == kStagesBwd - 1 ? 0 : slot + 1;
  }
  if (p.dh0 != nullptr && rank == 0 && tid < 16)
    store_row<float, VEC>(p.dh0 + static_cast<int64_t>(b) * D, c0, lane, D, carry);
}

template <typename E, int G>
__global__ void __launch_bounds__(256) scan_step_kernel(float* __restrict__ h,
                                                        const E* __restrict__ x,
                                                        const E* __restrict__ g, int64_t n,
                                                        E* __restrict__ y) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float a, keep;
  gate<G>(load_as_float(g + i), a, keep);
  const float v = fmaf(a, h[i], keep * load_as_float(x + i));
  h[i] = v;
  y[i] = store_from_float<E>(v);
}

// CTAs of a cluster: enough of them for two on every SM, as far as the sequence
// has tiles for them.
int cluster_of(int64_t units, int tiles) {
  int n = 1;
  while (n < kMaxCluster && n < tiles && units * n < 2 * 152) n *= 2;
  return n;
}

template <typename Args>
cudaError_t launch(void (*kernel)(Args, int, int), const Args& a, int tile, int bytes,
                   cudaStream_t st) {
  const int blocks = (a.D + kChannels - 1) / kChannels;
  const int64_t units = static_cast<int64_t>(a.B) * blocks;
  const int n = cluster_of(units, (a.T + tile - 1) / tile);
  if (bytes > 0) {
    const cudaError_t e = cudaFuncSetAttribute(
        reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * n));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, blocks, n);
}

template <typename E, int G, bool VEC>
cudaError_t fwd_of(const ScanArgs& a, cudaStream_t st) {
  return launch<ScanArgs>(scan_fwd_kernel<E, G, VEC>, a, kRuns * kRunFwd<E>,
                          Tiles<E, VEC, 2, kRunFwd<E>, kStagesFwd>::kBytes, st);
}
template <typename E, int G>
cudaError_t fwd(const ScanArgs& a, cudaStream_t st) {
  return a.D % 4 == 0 ? fwd_of<E, G, true>(a, st) : fwd_of<E, G, false>(a, st);
}

template <typename E, int G, bool VEC>
cudaError_t bwd_of(const ScanBwdArgs& a, cudaStream_t st) {
  return launch<ScanBwdArgs>(scan_bwd_kernel<E, G, VEC>, a, kMark,
                             Tiles<E, VEC, 3, kRunBwd, kStagesBwd>::kBytes, st);
}
template <typename E, int G>
cudaError_t bwd(const ScanBwdArgs& a, cudaStream_t st) {
  return a.D % 4 == 0 ? bwd_of<E, G, true>(a, st) : bwd_of<E, G, false>(a, st);
}

template <typename E, int G>
cudaError_t step(float* h, const void* x, const void* g, int64_t n, void* y, cudaStream_t st) {
  scan_step_kernel<E, G><<<static_cast<unsigned>((n + 255) / 256), 256, 0, st>>>(
      h, static_cast<const E*>(x), static_cast<const E*>(g), n, static_cast<E*>(y));
  return cudaGetLastError();
}

}  // namespace

cudaError_t gated_scan_fwd_launch(const ScanArgs& a, cudaStream_t st) {
  using B16 = __nv_bfloat16;
  if (a.dtype == SANATAN_F32)
    return a.gate == SANATAN_GATE_LOG ? fwd<float, SANATAN_GATE_LOG>(a, st)
                                      : fwd<float, SANATAN_GATE_SIGMOID>(a, st);
  return a.gate == SANATAN_GATE_LOG ? fwd<B16, SANATAN_GATE_LOG>(a, st)
                                    : fwd<B16, SANATAN_GATE_SIGMOID>(a, st);
}

cudaError_t gated_scan_bwd_launch(const ScanBwdArgs& a, cudaStream_t st) {
  using B16 = __nv_bfloat16;
  if (a.dtype == SANATAN_F32)
    return a.gate == SANATAN_GATE_LOG ? bwd<float, SANATAN_GATE_LOG>(a, st)
                                      : bwd<float, SANATAN_GATE_SIGMOID>(a, st);
  return a.gate == SANATAN_GATE_LOG ? bwd<B16, SANATAN_GATE_LOG>(a, st)
                                    : bwd<B16, SANATAN_GATE_SIGMOID>(a, st);
}

cudaError_t gated_scan_step_launch(float* h, const void* x, const void* g, int dtype, int gate,
                                   int64_t n, void* y, cudaStream_t st) {
  using B16 = __nv_bfloat16;
  if (dtype == SANATAN_F32)
    return gate == SANATAN_GATE_LOG ? step<float, SANATAN_GATE_LOG>(h, x, g, n, y, st)
                                    : step<float, SANATAN_GATE_SIGMOID>(h, x, g, n, y, st);
  return gate == SANATAN_GATE_LOG ? step<B16, SANATAN_GATE_LOG>(h, x, g, n, y, st)
                                  : step<B16, SANATAN_GATE_SIGMOID>(h, x, g, n, y, st);
}

}  // namespace sanatan
