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
// Four warps walk 128 / L channels of a stretch of tokens, L lanes a channel, four states a
// lane (L = N / 4, up to a power of two, 4 at least); neighbouring lanes have neighbouring
// channels, so that loads of B and C from shared memory, the same for both, are half as long.
// Tiles of sixteen tokens are copied to shared memory ahead; delta, delta u and v are formed
// once for each token and channel and left there with B and C; then each lane walks its four
// states through the tile.  Sums over the states meet by shuffles, four tokens at a time, so
// that a lane ends with one finished sum; sums over channels (dB, dC) likewise, then over the
// warps in shared memory.
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
//
// Bound: instructions and their latency, not bytes.  A token, channel and state costs one
// exponential and eight other operations forward, an exponential and a half and about
// twenty-five backward, packed two an instruction, beside what a token and channel costs
// once (a softplus and the gate).  GB300, N 16, bf16, gated: B 8 T 4096 D 1536
// forward 425 us (440 with marks; 0.8 G states, 1.9 T a second; the bytes alone would take 61),
// backward 1390 (the bytes 106); B 1 T 32768 D 1536 597 and 1452 (segments walk twice).  First
// version (loads by the element, decays by the series, 2 barriers a tile): 1540 and 4000.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "copy_async.cuh"
#include "f32x2.cuh"
#include "fast_math.cuh"
#include "pdl.cuh"
#include "sanatan_internal.h"
#include "sanatan_math.cuh"
#include "vec_io.cuh"

namespace sanatan {
namespace {

using namespace f2;

constexpr int kTile = kSelectiveMark;  // tokens of a tile, and between two marks
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStates = 4;             // of a lane
constexpr int kSegmentLanes = 16;      // more lanes a channel: never cut into segments
constexpr float kLn2 = 0.6931471805599453f;

template <int L>
struct Geo {
  static constexpr int CW = 32 / L;          // channels of a warp
  static constexpr int CB = CW * kWarps;     // of a block
  static constexpr int NP = kStates * L;     // states, with those that fill up
  // A warp's cells, (token, channel) pairs of a tile: a lane has one token of W neighbouring
  // channels; where that makes sixteen lanes, the others have none.
  static constexpr int W = CW < 4 ? CW : 4;
  static constexpr bool kAllLanes = CW / W == 2;
  static constexpr int kRowPitch = CW + 1;                 // of float4: no bank conflicts
  // B and C of a tile, four states at a time: quads of a thread.
  static constexpr int kQuadItems = kTile * 2 * L / kThreads;
  static_assert(L >= 4 && kTile * CW / W <= 32 && kTile * 2 * L % kThreads == 0);
};

__device__ __forceinline__ float sum2(uint64_t v) {
  float a, b;
  upk2(v, a, b);
  return a + b;
}
// 2^x of a pair by the hardware, which is 0.1 to 0.8 steps of 2^-24 low on average (measured,
// by binades of x).  A memory of n tokens multiplies that by n: see Decays.
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) {
  float a, b;
  upk2(x, a, b);
  return pk2(ex2(a), ex2(b));
}

// 2^x without that bias where x is small: the first four terms of the series are within 0.15
// steps for |x| < 1/32 (x ln 2 < 0.0217; the next is its fourth power / 24).
__device__ __forceinline__ float exp2_near(float x) {
  const float p = fmaf(fmaf(fmaf(0.055504108664821580f, x, 0.24022650695910072f), x, kLn2), x,
                       1.0f);  // (ln(2)^3 / 6, ln(2)^2 / 2, ln(2))
  return fabsf(x) < 0.03125f ? p : ex2(x);
}

// What the decays of a tile multiply a lane's states by: their product as they were rounded,
// and the sum of delta, which gives what it should be, 2^(A sum delta).  Their ratio puts
// the state right once a tile, so that the bias of sixteen decays (at most 16 x 0.8 steps, 8e-7)
// is all that is ever in a state, whatever its memory.  (The series for every decay instead:
// 973 us for the forward of B 8 T 4096 D 1536 N 16 bf16, 750 so.)
//
// Steps of both signs (without a softplus): a product may leave float32, or lose its digits
// among its smallest numbers, and come back though the sum is small.  What a product reaches
// on the way is at most 2^(|A| sum |delta|): where that is large the state stays as walked.
struct Decays {
  uint64_t q0, q1, sum;
  __device__ __forceinline__ Decays() : q0(pk2(1.0f, 1.0f)), q1(q0), sum(pk2(0.0f, 0.0f)) {}
  __device__ __forceinline__ void add(uint64_t a0, uint64_t a1, uint64_t delta) {
    q0 = fmul2(q0, a0), q1 = fmul2(q1, a1), sum = fadd2(sum, delta);
  }
  // (a reach |A| sum |delta| of 8 and more: the memory is two tokens, or q may have no digits)
  __device__ __forceinline__ static float ratio(float x, float reach, float q) {
    return fabsf(reach) < 8.0f ? exp2_near(x) * rcp(q) : 1.0f;
  }
  // cells: the tile's, of the lane's channel, `pitch` apart, delta first.
  __device__ __forceinline__ void put_right(uint64_t A0, uint64_t A1, uint64_t& h0, uint64_t& h1,
                                            bool soft, const float4* cells, int pitch) const {
    float x[kStates], q[kStates], reach[kStates];
    upk2(fmul2(sum, A0), x[0], x[1]);
    upk2(fmul2(sum, A1), x[2], x[3]);
#pragma unroll
    for (int j = 0; j < kStates; ++j) reach[j] = x[j];  // (of a softplus: no step is negative)
    if (!soft) {
      float s = 0.0f;
#pragma unroll 1
      for (int t = 0; t < kTile; ++t) s += fabsf(cells[t * pitch].x);
      upk2(fmul2(pk2(s, s), A0), reach[0], reach[1]);
      upk2(fmul2(pk2(s, s), A1), reach[2], reach[3]);
    }
    upk2(q0, q[0], q[1]);
    upk2(q1, q[2], q[3]);
    h0 = fmul2(h0, pk2(ratio(x[0], reach[0], q[0]), ratio(x[1], reach[1], q[1])));
    h1 = fmul2(h1, pk2(ratio(x[2], reach[2], q[2]), ratio(x[3], reach[3], q[3])));
  }
};

// log(1 + exp(x)) = max(x, 0) + log(1 + e) of a pair, e = exp(-|x|) <= 1, with log(1 + e) = 2
// atanh(r), r = e / (2 + e) <= 1/3: the series r + r^3 / 3 + r^5 / 5 ... to r^13 is within
// 2^-26 of its value, for all e alike.  A small step has e's own error, the rounding of
// |x| log2(e): |x| 2^-24 of itself, 4e-7 for a delta of 0.001.
__device__ __forceinline__ uint64_t softplus_pair(uint64_t x) {
  float x0, x1, e0, e1;
  upk2(x, x0, x1);
  e0 = ex2(fabsf(x0) * -kLog2e), e1 = ex2(fabsf(x1) * -kLog2e);
  const uint64_t r = pk2(e0 * rcp(2.0f + e0), e1 * rcp(2.0f + e1));
  const uint64_t q = fmul2(r, r);
  auto both = [](float c) { return pk2(c, c); };
  uint64_t p = ffma2(q, both(1.0f / 13), both(1.0f / 11));
  p = ffma2(p, q, both(1.0f / 9));
  p = ffma2(p, q, both(1.0f / 7));
  p = ffma2(p, q, both(1.0f / 5));
  p = ffma2(p, q, both(1.0f / 3));
  p = ffma2(p, q, both(1.0f));
  // (a NaN goes through r; fmaxf alone would drop it)
  return ffma2(fmul2(r, both(2.0f)), p, pk2(fmaxf(x0, 0.0f), fmaxf(x1, 0.0f)));
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
  int b, seg, cb, tiles, k0, k1;  // k0 .. k1: the segment's tiles
  __device__ __forceinline__ Place(const SelectiveArgs& a) {
    cb = blockIdx.x % a.blocks;
    const unsigned rest = blockIdx.x / a.blocks;
    seg = rest % a.segments;
    b = rest / a.segments;
    tiles = (a.T + kTile - 1) / kTile;
    k0 = seg * a.tiles_per_segment;
    k1 = min(k0 + a.tiles_per_segment, tiles);
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

// A tile of the tensors of a block, as they are in memory, on its way to shared memory while
// tiles before are worked on: NT tensors of [B, T, D] (its channels), then B and C.  Where
// rows are words, by asynchronous copies, the same few places of every tile for a thread;
// else through registers (begin() loads, end() stores).  Tokens behind the sequence and
// channels behind the last are zeros, and not read.
template <typename E, int L, bool ALIGNED, int NT>
struct Stage {
  using G = Geo<L>;
  static constexpr int kSize = sizeof(E);
  static constexpr int kRow = G::CB * kSize;                 // bytes
  static constexpr int kChunk = kRow < 16 ? kRow : 16;
  static constexpr int kPitch = kRow + 16;                   // (rows in different banks)
  static constexpr int kCell = kTile * kPitch;
  static constexpr int kPairPitch = G::NP * kSize;
  static constexpr int kPair = kTile * kPairPitch;
  static constexpr int kBytes = NT * kCell + 2 * kPair;      // of a buffer
  static constexpr int kPer = kRow / kChunk, kCellChunks = kTile * kPer;
  static constexpr int kPairPer = (kPairPitch + 15) / 16, kPairChunks = kTile * kPairPer;
  static constexpr int kChunks = NT * kCellChunks + 2 * kPairChunks;
  static constexpr int kSlots = ALIGNED ? (kChunks + kThreads - 1) / kThreads : 1;
  static constexpr int kOne = kTile * G::CB / kThreads > 0 ? kTile * G::CB / kThreads : 1;
  static constexpr int kPairOne = kTile * G::NP / kThreads > 0 ? kTile * G::NP / kThreads : 1;
  static constexpr int kNever = 1 << 30;

  // ALIGNED: where a slot's next copy comes from and goes to, its token of the tile
  const char* from[kSlots];
  int64_t step[kSlots];
  int to[kSlots], token[kSlots], bytes[kSlots];
  // else: what is on its way
  E r[ALIGNED ? 1 : NT * kOne + 2 * kPairOne];
  const E* x[NT + 2];
  int64_t ld[NT + 2], row0;
  int n, d0, D, N;

  // A null tensor is left out.  Tiles go from k on, up (dir 1) or down (-1).
  __device__ __forceinline__ void init(const void* const (&tensors)[NT + 2],
                                       const int64_t (&lds)[NT + 2], const SelectiveArgs& a,
                                       int64_t row0_, int n_, int d0_, int k, int dir) {
    n = n_, d0 = d0_, D = a.D, N = a.N, row0 = row0_;
#pragma unroll
    for (int q = 0; q < NT + 2; ++q) x[q] = static_cast<const E*>(tensors[q]), ld[q] = lds[q];
    if constexpr (ALIGNED) place(a, k, dir);
  }
  __device__ __forceinline__ void place(const SelectiveArgs& a, int k, int dir) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      int c = threadIdx.x % kThreads + i * kThreads;
      from[i] = reinterpret_cast<const char*>(x[0]);
      step[i] = 0, to[i] = 0, token[i] = kNever, bytes[i] = 0;
      int base = 0;
#pragma unroll
      for (int q = 0; q < NT + 2; ++q) {
        const bool cell = q < NT;
        const int chunks = cell ? kCellChunks : kPairChunks, per = cell ? kPer : kPairPer;
        const int chunk = cell ? kChunk : 16;
        if (c >= 0 && c < chunks) {
          const int t = c / per, at = c % per * chunk, v = at / kSize;
          to[i] = base + t * (cell ? kPitch : kPairPitch) + at;
          bytes[i] = chunk;
          if (x[q] != nullptr && (cell ? d0 + v < D : v < N)) {
            from[i] = reinterpret_cast<const char*>(
                x[q] + (row0 + static_cast<int64_t>(k) * kTile + t) * ld[q] + (cell ? d0 + v : v));
            step[i] = ld[q] * (dir * kTile * kSize);
            token[i] = t;
          }
        }
        c -= chunks;
        base += cell ? kCell : kPair;
      }
    }
  }
  __device__ __forceinline__ void begin(char* buffer, int k) {
    const int left = n - k * kTile;
    if constexpr (ALIGNED) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        // (a place without a token reads nothing, and from no address outside the tensor)
        const bool real = token[i] < left;
        const void* source = real ? from[i] : reinterpret_cast<const char*>(x[0]);
        if (kChunk == 16) {
          if (i + 1 < kSlots || kChunks % kThreads == 0 || bytes[i] != 0)
            copy_or_zeros(buffer + to[i], source, real, 16);
        } else if (bytes[i] == 16) {
          copy_or_zeros(buffer + to[i], source, real, 16);
        } else if (bytes[i] != 0) {
          copy_or_zeros(buffer + to[i], source, real, kChunk);
        }
        from[i] += step[i];
      }
      copy_commit();
    } else {
      load(row0 + static_cast<int64_t>(k) * kTile, left);
    }
  }
  __device__ __forceinline__ void load(int64_t row, int left) {
#pragma unroll
    for (int q = 0; q < NT + 2; ++q) {
      if (x[q] == nullptr) continue;
#pragma unroll
      for (int i = 0; i < (q < NT ? kOne : kPairOne); ++i) {
        const int c = threadIdx.x % kThreads + i * kThreads;
        const int t = q < NT ? c / G::CB : c / G::NP, v = q < NT ? d0 + c % G::CB : c % G::NP;
        const bool real = t < kTile && t < left && v < (q < NT ? D : N);
        // (one load whether real or not: a branch would wait for it)
        E e = *(real ? x[q] + (row + t) * ld[q] + v : x[q]);
        if (!real) e = store_from_float<E>(0.0f);
        r[(q < NT ? q * kOne : NT * kOne + (q - NT) * kPairOne) + i] = e;
      }
    }
  }
  __device__ __forceinline__ void end(char* buffer) const {
    if constexpr (!ALIGNED) store(buffer);
  }
  __device__ __forceinline__ void store(char* buffer) const {
#pragma unroll
    for (int q = 0; q < NT + 2; ++q) {
      if (x[q] == nullptr) continue;
      char* base = buffer + (q < NT ? q * kCell : NT * kCell + (q - NT) * kPair);
#pragma unroll
      for (int i = 0; i < (q < NT ? kOne : kPairOne); ++i) {
        const int c = threadIdx.x % kThreads + i * kThreads;
        const int t = q < NT ? c / G::CB : c / G::NP, v = q < NT ? c % G::CB : c % G::NP;
        if (t < kTile)
          *reinterpret_cast<E*>(base + t * (q < NT ? kPitch : kPairPitch) + v * kSize) =
              r[(q < NT ? q * kOne : NT * kOne + (q - NT) * kPairOne) + i];
      }
    }
  }
  // W channels of a token of tensor q from c, as floats.
  __device__ __forceinline__ static void get(const char* buffer, int q, int t, int c,
                                             float (&f)[G::W]) {
    Vec<E, G::W> v;
    v.load(reinterpret_cast<const E*>(buffer + q * kCell + t * kPitch + c * kSize));
    v.get(f);
  }
  // B and C from there to floats, [token][B | C][ORDERS][WIDE], zeros behind N.
  template <int ORDERS, int WIDE>
  __device__ __forceinline__ static void pairs_to_float(const char* buffer, int N,
                                                        float (*pairs)[2][ORDERS][WIDE]);
};

// The order of a lane's states in its registers: register j holds state j ^ order.  In the
// backward's main kernel neighbouring channels hold theirs in different orders, so that where
// two lanes halve their values each keeps the first and sends the last, without selecting.
__device__ __forceinline__ void reorder(float (&f)[kStates], int order) {
  if (order & 2) {
    const float a = f[0], b = f[1];
    f[0] = f[2], f[1] = f[3], f[2] = a, f[3] = b;
  }
  if (order & 1) {
    const float a = f[0], b = f[2];
    f[0] = f[1], f[2] = f[3], f[1] = a, f[3] = b;
  }
}

template <typename E, int L, bool ALIGNED, int NT>
template <int ORDERS, int WIDE>
__device__ __forceinline__ void Stage<E, L, ALIGNED, NT>::pairs_to_float(
    const char* buffer, int N, float (*pairs)[2][ORDERS][WIDE]) {
#pragma unroll
  for (int i = 0; i < G::kQuadItems; ++i) {
    const int k = threadIdx.x % kThreads + i * kThreads;
    const int q = k % L, which = k / L % 2, t = k / (2 * L);
    Vec<E, 4> v;
    float f[4];
    v.load(reinterpret_cast<const E*>(buffer + NT * kCell + which * kPair + t * kPairPitch) +
           4 * q);
    v.get(f);
    if (4 * q + 4 > N)  // (what fills up a row of B or C need not be zero)
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = 4 * q + j < N ? f[j] : 0.0f;
#pragma unroll
    for (int o = 0; o < ORDERS; ++o) {
      const int x = (o & 1) * 2 + (o >> 1);
      *reinterpret_cast<float4*>(&pairs[t][which][o][4 * q]) =
          make_float4(f[0 ^ x], f[1 ^ x], f[2 ^ x], f[3 ^ x]);
    }
  }
}

// delta of W cells of a token from dt (zero where the token is not there: a = 1 and no
// input, the state passes).
template <int W>
__device__ __forceinline__ void steps(float (&delta)[W], const float (&bias)[W], bool soft,
                                      bool real) {
#pragma unroll
  for (int j = 0; j < W; ++j) delta[j] += bias[j];
  if (soft) {
#pragma unroll
    for (int j = 0; j < W; j += 2) {
      float other = 0.0f;
      upk2(softplus_pair(pk2(delta[j], delta[j + 1 < W ? j + 1 : j])), delta[j],
           j + 1 < W ? delta[j + 1] : other);
    }
  }
#pragma unroll
  for (int j = 0; j < W; ++j) delta[j] = real ? delta[j] : 0.0f;
}

// W neighbours of a row from d, those that exist.
template <typename E, int W, bool ALIGNED>
__device__ __forceinline__ void store_cells(E* row, int d, int D, const float (&f)[W]) {
  if (ALIGNED) {
    Vec<E, W> v;
    v.put(f);
    if (d < D) v.store(row + d);
  } else {
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (d + j < D) row[d + j] = store_from_float<E>(f[j]);
  }
}

// decay h + own for a decay of 2^x.  A segment's decay may be outside float32 where no state
// is: its fourth root is multiplied in step by step there, and nothing makes nothing of it.
__device__ __forceinline__ float carried(float x, float h, float own) {
  if (fabsf(x) < 126.0f) return fmaf(ex2(x), h, own);
  const float root = ex2(0.25f * x);
  return h == 0.0f ? own : fmaf(h * root * root * root, root, own);
}

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
  constexpr int kAhead = 4;  // segments whose loads are under way together
  for (int k = 0; k < S; k += kAhead) {
    float own[kAhead], x[kAhead];
    int64_t s[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k + j < S) {
        s[j] = b * S + (reverse ? S - 1 - k - j : k + j);
        own[j] = H[s[j] * slab + at], x[j] = a * sums[s[j] * D + d];
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k + j < S) {
        H[s[j] * slab + at] = h;
        h = carried(x[j], h, own[j]);
      }
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
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), threads, shared, st, args...);
}

cudaError_t launch_carry(const SelectiveArgs& a, const float* first, bool reverse,
                         cudaStream_t st) {
  const int64_t all = static_cast<int64_t>(a.B) * a.D * a.N;
  return launch(selective_carry_kernel, (all - 1) / 256 + 1, 256, 0, st, a.carry,
                static_cast<const float*>(a.sums), a.A, first, a.segments, a.D, a.N, all, reverse);
}

// Whether every row of every tensor is 16-byte words.
template <typename E>
bool words(const SelectiveArgs& a, std::initializer_list<const void*> dense) {
  const int64_t V = 16 / sizeof(E);
  if (a.D % V != 0 || a.N % V != 0 || a.ldb % V != 0 || a.ldc % V != 0) return false;
  if (a.z != nullptr && a.ldz % V != 0) return false;
  for (const void* p : {a.u, a.dt, a.z, a.Bm, a.Cm})
    if (!at_bytes(p, 16)) return false;
  for (const void* p : dense)
    if (!at_bytes(p, 16)) return false;
  return true;
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
