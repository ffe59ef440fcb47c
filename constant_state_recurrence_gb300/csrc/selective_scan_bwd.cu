// The selective scan's backward (formulas and method: selective_scan.cuh).
//
// A tile is walked forward from its mark to the states before every fourth token, which are put
// aside, then back by fours: decays and states of four tokens are formed again, then their
// gradients.  Bound: instructions, 129 a token and warp (a quarter of them the sums over
// channels and states), half of the issue slots used by the ten warps that an SM has at the
// training shape.  With all decays of a tile in registers and all states in shared memory it was
// the latter's wavefronts, 42 a token and warp: 1466 us instead of 1422 then (1390 now), one
// prompt of 32768 tokens 1840 instead of 1567 (1452 now).  Cells as pairs twice over, without the
// moves that make pairs of them: 1563.
//
// dB and dC are sums over channels: each block of 128 / L channels leaves its part of them for
// every token, in all L / 4 times the marks.  Beyond four lanes a channel and 512 MB the parts
// are kept no larger than the marks: segments are walked in pieces, from the last, by a launch
// each that takes all segments, with the gradient behind a piece and the sums over tokens in
// memory between two (so that nothing is added in another order), and a piece's parts are
// added up before the next overwrites them.  B 4 T 4096 D 4096 N 128 bf16: 17.2 GB and 18.8 ms
// in one piece, 2.2 GB and 19.3 ms in eight; B 1 T 4096 D 1536 N 128: 1.6 GB and 2.57 ms, 0.54
// and 2.75 in three.
#include "selective_scan.cuh"

namespace sanatan {
namespace {

template <typename E, int L, bool ALIGNED>
struct BwdStateShared {
  using G = Geo<L>;
  using Tiles = Stage<E, L, ALIGNED, 3>;      // dt, z, dy
  float4 cells[kWarps][kTile][G::kRowPitch];  // delta, delta, v, v
  float pairs[2][kTile][2][1][G::NP];
  char raw[3][Tiles::kBytes];
};

// The walk back alone, from no gradient behind the segment: what its own tokens add to the
// gradient before it, and its sum of delta.
template <typename E, int L, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) selective_bwd_state_kernel(SelectiveBwdArgs args) {
  using G = Geo<L>;
  constexpr int W = G::W;
  using Sm = BwdStateShared<E, L, ALIGNED>;
  using Tiles = typename Sm::Tiles;
  const SelectiveArgs& a = args.f;
  extern __shared__ float4 smem4[];
  Sm& sm = *reinterpret_cast<Sm*>(smem4);
  const Place<L> at(a);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, l = lane / G::CW;
  const int mine = lane % G::CW;
  const int d0 = at.cb * G::CB, w0 = d0 + warp * G::CW, d = w0 + mine;
  constexpr int kPer = G::CW / W;
  const int cell_c = lane % kPer * W, cell_t = lane / kPer, cell_d = w0 + cell_c;
  const StatePlace st(d, l, a.D, a.N, a.vec);
  wait_for_previous();
  const int n = length_of(a.lens, at.b, a.T);
  const int64_t slab = static_cast<int64_t>(a.D) * a.N, row0 = static_cast<int64_t>(at.b) * a.T;
  const bool gated = a.z != nullptr;
  const int live = min(at.k1, (n + kTile - 1) / kTile), last = live - 1;
  Tiles tiles;
  tiles.init({a.dt, a.z, args.dy, nullptr, a.Cm}, {a.D, a.ldz, a.D, 0, a.ldc}, a, row0, n, d0,
             last, -1);
  if (last >= at.k0) tiles.begin(sm.raw[0], last), tiles.end(sm.raw[0]);
  if (last > at.k0) tiles.begin(sm.raw[1], last - 1), tiles.end(sm.raw[1]);
  float f[kStates];
  st.load(a.A, f);
  const uint64_t A0 = pk2(f[0] * kLog2e, f[1] * kLog2e), A1 = pk2(f[2] * kLog2e, f[3] * kLog2e);
  uint64_t g0 = pk2(0.0f, 0.0f), g1 = g0;
  float bias[W], sum[W];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    bias[j] = cell_d + j < a.D && a.dt_bias != nullptr ? a.dt_bias[cell_d + j] : 0.0f;
    sum[j] = 0.0f;
  }
  if (last >= at.k0) {
    copy_wait<0>();
    __syncthreads();
    Tiles::pairs_to_float(sm.raw[0], a.N, sm.pairs[last & 1]);
  }
  int now = 0;  // the buffer of tile k
  for (int k = last; k >= at.k0; --k) {
    const int next = now == 2 ? 0 : now + 1, after = next == 2 ? 0 : next + 1;
    copy_wait<0>();
    __syncthreads();
    if (k - 2 >= at.k0) tiles.begin(sm.raw[after], k - 2);
    if (k > at.k0) Tiles::pairs_to_float(sm.raw[next], a.N, sm.pairs[(k - 1) & 1]);
    if (G::kAllLanes || cell_t < kTile) {
      const int t = cell_t;
      float delta[W], v[W], z[W];
      Tiles::get(sm.raw[now], 0, t, warp * G::CW + cell_c, delta);
      Tiles::get(sm.raw[now], 2, t, warp * G::CW + cell_c, v);
      if (gated) Tiles::get(sm.raw[now], 1, t, warp * G::CW + cell_c, z);
      steps<W>(delta, bias, a.softplus, k * kTile + t < n);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        sum[j] += delta[j];
        if (gated) v[j] *= z[j] * sigmoid(z[j]);
        sm.cells[warp][t][cell_c + j] = make_float4(delta[j], delta[j], v[j], v[j]);
      }
    }
    __syncwarp();
    Decays decays;
#pragma unroll
    for (int t = kTile - 1; t >= 0; --t) {
      const ulonglong2 c = reinterpret_cast<const ulonglong2&>(sm.cells[warp][t][mine]);
      const ulonglong2 Cv =
          reinterpret_cast<const ulonglong2&>(sm.pairs[k & 1][t][1][0][kStates * l]);
      const uint64_t a0 = exp2_pair(fmul2(c.x, A0)), a1 = exp2_pair(fmul2(c.x, A1));
      g0 = fmul2(a0, ffma2(c.y, Cv.x, g0));
      g1 = fmul2(a1, ffma2(c.y, Cv.y, g1));
      decays.add(a0, a1, c.x);
    }
    decays.put_right(A0, A1, g0, g1, a.softplus, &sm.cells[warp][0][mine], G::kRowPitch);
    __syncwarp();
    if (k - 2 >= at.k0) tiles.end(sm.raw[after]);
    now = next;
  }
  const int64_t part = static_cast<int64_t>(at.b) * a.segments + at.seg;
  st.store(a.carry + part * slab, g0, g1);
#pragma unroll
  for (int j = 0; j < W; ++j) {
#pragma unroll
    for (int bit = kPer; bit < 32; bit *= 2) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], bit);
    if (cell_t == 0 && cell_d + j < a.D) a.sums[part * a.D + cell_d + j] = sum[j];
  }
}

// The lane bits over which the sums over channels are halved: first by two states of four,
// then by one of two, so that these say a lane's order; then (where there is a third) into
// dB and dC.  Neighbouring lanes have the same order where they can.
template <int L>
struct Bits {
  static constexpr int CW = Geo<L>::CW;
  static constexpr int A = CW >= 4 ? 2 : 1, B = CW >= 8 ? 4 : 1;  // (dB and dC: 1)
  static constexpr int kOrders = CW < 4 ? CW : 4;
  __device__ __forceinline__ static int order(int lane) {  // 0 .. kOrders - 1
    return (CW >= 2 && (lane & A) ? 1 : 0) + (CW >= 4 && (lane & B) ? 2 : 0);
  }
};

template <typename E, int L, bool ALIGNED>
struct BwdShared {
  using G = Geo<L>;
  using Tiles = Stage<E, L, ALIGNED, 4>;      // u, dt, z, dy
  float4 states[kWarps][kTile / 4][32];       // of each lane, before every fourth token
  float by_warp[kWarps][kTile][2][G::NP];     // a warp's sums of dB and dC
  float4 cells[kWarps][kTile][G::kRowPitch];  // delta, delta u, v, v
  float pairs[kTile][2][Bits<L>::kOrders][G::NP + 8];  // (orders in different banks)
  float sums[kWarps][3][kTile][G::CW];        // of dh B, of w A, and y
  char raw[Tiles::kBytes];
};

__device__ __forceinline__ uint64_t shfl2(uint64_t v, int bit) {
  float a, b;
  upk2(v, a, b);
  return pk2(__shfl_xor_sync(0xffffffffu, a, bit), __shfl_xor_sync(0xffffffffu, b, bit));
}

// The sum over a warp's channels of its lanes' dB and dC (b0: registers 0 and 1, b1: 2 and
// 3).  Returns how a lane's values are to be written: out [0], or [0] (dB) and [1] (dC), or
// [0, 1] and [2, 3], or all eight.
template <int L>
__device__ __forceinline__ void sum_channels(uint64_t b0, uint64_t b1, uint64_t c0, uint64_t c1,
                                             int lane, float (&out)[8]) {
  constexpr int CW = Geo<L>::CW;
  if constexpr (CW >= 2) {
    b0 = fadd2(b0, shfl2(b1, Bits<L>::A));
    c0 = fadd2(c0, shfl2(c1, Bits<L>::A));
    float p, q, r, s;
    upk2(b0, p, q);
    upk2(c0, r, s);
    if constexpr (CW >= 4) {
      p += __shfl_xor_sync(0xffffffffu, q, Bits<L>::B);
      r += __shfl_xor_sync(0xffffffffu, s, Bits<L>::B);
      if constexpr (CW == 8) {
        const bool up = lane & 1;
        p = (up ? r : p) + __shfl_xor_sync(0xffffffffu, up ? p : r, 1);
      }
    }
    out[0] = p, out[1] = CW >= 4 ? r : q, out[2] = r, out[3] = s;
  } else {
    upk2(b0, out[0], out[1]);
    upk2(b1, out[2], out[3]);
    upk2(c0, out[4], out[5]);
    upk2(c1, out[6], out[7]);
  }
}
// They go to [B | C][NP] of the token; x: the lane's order.
template <int L>
__device__ __forceinline__ void put_channels(const float (&v)[8], int lane, int x, float* to) {
  constexpr int CW = Geo<L>::CW, NP = Geo<L>::NP;
  float* at = to + kStates * (lane / CW);
  if constexpr (CW == 8) {
    at[(lane & 1) * NP + x] = v[0];
  } else if constexpr (CW == 4) {
    at[x] = v[0];
    at[NP + x] = v[1];
  } else if constexpr (CW == 2) {
    at[0 ^ x] = v[0], at[1 ^ x] = v[1];
    at[NP + (0 ^ x)] = v[2], at[NP + (1 ^ x)] = v[3];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] = v[j], at[NP + j] = v[4 + j];
  }
}

template <typename E, int L, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, L == 4 ? 3 : 1)
    selective_bwd_kernel(SelectiveBwdArgs args) {
  using G = Geo<L>;
  constexpr int W = G::W;
  using Sm = BwdShared<E, L, ALIGNED>;
  using Tiles = typename Sm::Tiles;
  const SelectiveArgs& a = args.f;
  extern __shared__ float4 smem4[];
  Sm& sm = *reinterpret_cast<Sm*>(smem4);
  const Place<L> at(a);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, l = lane / G::CW;
  const int mine = lane % G::CW;
  const int d0 = at.cb * G::CB, w0 = d0 + warp * G::CW, d = w0 + mine;
  constexpr int kPer = G::CW / W, kStep = 32 / kPer;
  const int cell_c = lane % kPer * W, cell_t = lane / kPer, cell_d = w0 + cell_c;
  const int order = Bits<L>::order(lane), x = (order & 1) * 2 + (order >> 1);
  const StatePlace st(d, l, a.D, a.N, a.vec);
  wait_for_previous();
  const int n = length_of(a.lens, at.b, a.T);
  const int64_t slab = static_cast<int64_t>(a.D) * a.N, row0 = static_cast<int64_t>(at.b) * a.T;
  const int64_t part = static_cast<int64_t>(at.b) * a.segments + at.seg;
  const bool gated = a.z != nullptr;
  E* DU = static_cast<E*>(args.du);
  E* DDT = static_cast<E*>(args.ddt);
  E* DZ = static_cast<E*>(args.dz);
  // The piece's tiles k0 .. k1 of the segment's (four lanes a channel: always all of them).
  constexpr bool kPieces = L > 4;
  const int k0 = kPieces ? min(at.k0 + args.piece * args.tiles_per_piece, at.k1) : at.k0;
  const int k1 = kPieces ? min(k0 + args.tiles_per_piece, at.k1) : at.k1;
  const bool first = !kPieces || args.piece + 1 == args.pieces, last = !kPieces || args.piece == 0;
  const int live = min(k1, (n + kTile - 1) / kTile);
  Tiles tiles;
  tiles.init({a.u, a.dt, a.z, args.dy, a.Bm, a.Cm}, {a.D, a.D, a.ldz, a.D, a.ldb, a.ldc}, a, row0,
             n, d0, live - 1, -1);
  float rmark[kStates];
  auto begin = [&](int k) {
    st.load(args.marks + (static_cast<int64_t>(at.b) * at.tiles + k) * slab, rmark);
    tiles.begin(sm.raw, k);
  };
  if (k0 < live) begin(live - 1), tiles.end(sm.raw);
  uint64_t A0, A1, g0, g1, dA0 = pk2(0.0f, 0.0f), dA1 = dA0;
  {
    float f[kStates];
    st.load(a.A, f);
    reorder(f, x);
    A0 = pk2(f[0] * kLog2e, f[1] * kLog2e), A1 = pk2(f[2] * kLog2e, f[3] * kLog2e);
    const float* from = a.segments > 1 || !first
                            ? a.carry + part * slab
                            : (args.dh_out != nullptr ? args.dh_out + at.b * slab : nullptr);
    f[0] = f[1] = f[2] = f[3] = 0.0f;
    if (from != nullptr) st.load(from, f);
    reorder(f, x);
    g0 = pk2(f[0], f[1]), g1 = pk2(f[2], f[3]);
    if (!first) {
      st.load(args.params + part * slab, f);
      reorder(f, x);
      dA0 = pk2(f[0], f[1]), dA1 = pk2(f[2], f[3]);
    }
  }
  float bias[W], skip[W], dskip[W], dbias[W];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const bool there = cell_d + j < a.D;
    bias[j] = there && a.dt_bias != nullptr ? a.dt_bias[cell_d + j] : 0.0f;
    skip[j] = there && a.skip != nullptr ? a.skip[cell_d + j] : 0.0f;
    dskip[j] = dbias[j] = 0.0f;
    if (!first && there && cell_t < kTile) {
      const float* from = args.lanes + (part * 2 * kTile + cell_t) * a.D + cell_d + j;
      dskip[j] = from[0], dbias[j] = from[static_cast<int64_t>(kTile) * a.D];
    }
  }
  {
    const float zero[W] = {};
    for (int t = max(k0, live) * kTile + cell_t; t < min(k1 * kTile, a.T); t += kStep) {
      store_cells<E, W, ALIGNED>(DU + (row0 + t) * a.D, cell_d, a.D, zero);  // without a token
      store_cells<E, W, ALIGNED>(DDT + (row0 + t) * a.D, cell_d, a.D, zero);
      if (gated) store_cells<E, W, ALIGNED>(DZ + (row0 + t) * a.D, cell_d, a.D, zero);
    }
  }
  // dB and dC of the block's channels and tile k: [block of channels][b][t][B | C][N], or
  // [block of channels][b][segment][t of the piece][B | C][N]
  auto put_pairs = [&](int k) {
    const int64_t rows = static_cast<int64_t>(args.tiles_per_piece) * kTile;
    const int64_t row = kPieces && args.pieces > 1
                            ? (static_cast<int64_t>(at.cb) * a.B * a.segments + part) * rows -
                                  static_cast<int64_t>(k0) * kTile
                            : static_cast<int64_t>(at.cb) * a.B * a.T + row0;
    float* out = args.pairs + row * 2 * a.N;
#pragma unroll
    for (int i = 0; i < G::kQuadItems; ++i) {
      const int q = tid + i * kThreads, s = q % L * 4, which = q / L % 2, tl = q / (2 * L);
      const int t = k * kTile + tl;
      if (t >= n || s >= a.N) continue;
      float sum[4] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v = reinterpret_cast<const float4&>(sm.by_warp[w][tl][which][s]);
        sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
      }
      float* o = out + (static_cast<int64_t>(t) * 2 + which) * a.N + s;
      if (a.N % 4 == 0 && a.vec) {
        *reinterpret_cast<float4*>(o) = make_float4(sum[0], sum[1], sum[2], sum[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (s + j < a.N) o[j] = sum[j];
      }
    }
  };
  for (int k = live - 1; k >= k0; --k) {
    copy_wait<0>();
    __syncthreads();
    if (k + 1 < live) put_pairs(k + 1);
    float u[W], raw[W], z[W], dy[W];
    if (G::kAllLanes || cell_t < kTile) {
      const int t = cell_t;
      const int c = warp * G::CW + cell_c;
      float delta[W];
      Tiles::get(sm.raw, 0, t, c, u);
      Tiles::get(sm.raw, 1, t, c, raw);
      if (gated) Tiles::get(sm.raw, 2, t, c, z);
      Tiles::get(sm.raw, 3, t, c, dy);
#pragma unroll
      for (int j = 0; j < W; ++j) delta[j] = raw[j];
      steps<W>(delta, bias, a.softplus, k * kTile + t < n);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float du = delta[j] * u[j];
        const float v = gated ? dy[j] * z[j] * sigmoid(z[j]) : dy[j];
        sm.cells[warp][t][cell_c + j] = make_float4(delta[j], du, v, v);
      }
    }
    Tiles::pairs_to_float(sm.raw, a.N, sm.pairs);
    reorder(rmark, x);
    uint64_t h0 = pk2(rmark[0], rmark[1]), h1 = pk2(rmark[2], rmark[3]);
    __syncthreads();
    if (k > k0) begin(k - 1);
    auto cell_of = [&](int t) { return sm.cells[warp][t][mine]; };
    auto pair_of = [&](int t, int which) {
      return reinterpret_cast<const ulonglong2&>(sm.pairs[t][which][order][kStates * l]);
    };
    // Forward to the state before every fourth token (a lane's own places).
    reinterpret_cast<ulonglong2&>(sm.states[warp][0][lane]) = make_ulonglong2(h0, h1);
#pragma unroll 1
    for (int g = 0; g < kTile - 4; g += 4) {
#pragma unroll
      for (int t = g; t < g + 4; ++t) {
        const float2 c = reinterpret_cast<const float2&>(sm.cells[warp][t][mine]);
        const uint64_t delta = pk2(c.x, c.x), du = pk2(c.y, c.y);
        const ulonglong2 Bv = pair_of(t, 0);
        h0 = ffma2(exp2_pair(fmul2(delta, A0)), h0, fmul2(du, Bv.x));
        h1 = ffma2(exp2_pair(fmul2(delta, A1)), h1, fmul2(du, Bv.y));
      }
      reinterpret_cast<ulonglong2&>(sm.states[warp][g / 4 + 1][lane]) = make_ulonglong2(h0, h1);
    }
    // Back by fours: the decays and states of four tokens, then their gradients.
    Decays decays;
#pragma unroll 1
    for (int g = kTile - 4; g >= 0; g -= 4) {
      float4 cell[4];
      uint64_t a[4][2], h[5][2];
      ulonglong2 Bv[4];
      const ulonglong2 before = reinterpret_cast<const ulonglong2&>(sm.states[warp][g / 4][lane]);
      h[0][0] = before.x, h[0][1] = before.y;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cell[i] = cell_of(g + i);
        Bv[i] = pair_of(g + i, 0);
        const uint64_t delta = pk2(cell[i].x, cell[i].x), du = pk2(cell[i].y, cell[i].y);
        a[i][0] = exp2_pair(fmul2(delta, A0)), a[i][1] = exp2_pair(fmul2(delta, A1));
        h[i + 1][0] = ffma2(a[i][0], h[i][0], fmul2(du, Bv[i].x));
        h[i + 1][1] = ffma2(a[i][1], h[i][1], fmul2(du, Bv[i].y));
        decays.add(a[i][0], a[i][1], delta);
      }
      float s[8], y[4];  // s: of dh B, then of w A, of four tokens
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const uint64_t delta = pk2(cell[i].x, cell[i].x), du = pk2(cell[i].y, cell[i].y);
        const uint64_t v = pk2(cell[i].z, cell[i].w);
        const ulonglong2 Cv = pair_of(g + i, 1);
        if (gated) y[i] = sum2(ffma2(h[i + 1][1], Cv.y, fmul2(h[i + 1][0], Cv.x)));
        const uint64_t dh0 = ffma2(v, Cv.x, g0), dh1 = ffma2(v, Cv.y, g1);
        g0 = fmul2(a[i][0], dh0), g1 = fmul2(a[i][1], dh1);
        const uint64_t w0 = fmul2(g0, h[i][0]), w1 = fmul2(g1, h[i][1]);
        dA0 = ffma2(w0, delta, dA0), dA1 = ffma2(w1, delta, dA1);
        s[i] = sum2(ffma2(dh1, Bv[i].y, fmul2(dh0, Bv[i].x)));
        s[4 + i] = sum2(ffma2(w1, A1, fmul2(w0, A0)));
        float p[8];
        sum_channels<L>(fmul2(du, dh0), fmul2(du, dh1), fmul2(v, h[i + 1][0]),
                        fmul2(v, h[i + 1][1]), lane, p);
        put_channels<L>(p, lane, x, &sm.by_warp[warp][g + i][0][0]);
      }
      if (gated) {
        using M = Meet<4, G::CW, 16>;
        M::sum(y, lane);
        if (M::first(lane))
#pragma unroll
          for (int q = 0; q < M::kLeft; ++q) sm.sums[warp][2][g + M::index(lane) + q][mine] = y[q];
      }
      using M = Meet<8, G::CW, 16>;
      M::sum(s, lane);
      if (M::first(lane))
#pragma unroll
        for (int q = 0; q < M::kLeft; ++q) {
          const int k8 = M::index(lane) + q;
          sm.sums[warp][k8 / 4][g + k8 % 4][mine] = s[q];
        }
    }
    decays.put_right(A0, A1, g0, g1, a.softplus, &sm.cells[warp][0][mine], G::kRowPitch);
    __syncwarp();
    if (G::kAllLanes || cell_t < kTile) {
      const int tl = cell_t, t = k * kTile + tl;
      float sB[W], sA[W], du[W], ddt[W], dz[W];
      Vec<float, W> r;
      r.load(&sm.sums[warp][0][tl][cell_c]);
      r.get(sB);
      r.load(&sm.sums[warp][1][tl][cell_c]);
      r.get(sA);
      if (gated) {
        r.load(&sm.sums[warp][2][tl][cell_c]);
        r.get(dz);
      }
      const bool real = t < n;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float4 cell = sm.cells[warp][tl][cell_c + j];
        const float delta = cell.x, v = cell.z;
        du[j] = fmaf(delta, sB[j], skip[j] * v);
        ddt[j] = fmaf(u[j], sB[j], sA[j] * kLn2);
        if (a.softplus) ddt[j] *= sigmoid(raw[j] + bias[j]);
        if (gated) {
          const float y0 = fmaf(skip[j], u[j], dz[j]), sg = sigmoid(z[j]);
          dz[j] = dy[j] * y0 * fmaf(z[j] * sg, 1.0f - sg, sg);
        }
        if (!real) du[j] = ddt[j] = dz[j] = 0.0f;
        dskip[j] = fmaf(v, u[j], dskip[j]);  // (zeros where there is no token)
        dbias[j] += ddt[j];
      }
      if (t < a.T) {
        store_cells<E, W, ALIGNED>(DU + (row0 + t) * a.D, cell_d, a.D, du);
        store_cells<E, W, ALIGNED>(DDT + (row0 + t) * a.D, cell_d, a.D, ddt);
        if (gated) store_cells<E, W, ALIGNED>(DZ + (row0 + t) * a.D, cell_d, a.D, dz);
      }
    }
    if (k > k0) tiles.end(sm.raw);
  }
  if (k0 < live) {
    __syncthreads();
    put_pairs(k0);
  }
  float f[kStates];
  float* to = !last ? a.carry + part * slab
                    : (args.dh0 != nullptr && at.seg == 0 ? args.dh0 + at.b * slab : nullptr);
  if (to != nullptr) {
    upk2(g0, f[0], f[1]);
    upk2(g1, f[2], f[3]);
    reorder(f, x);
    st.store(to, pk2(f[0], f[1]), pk2(f[2], f[3]));
  }
  upk2(dA0, f[0], f[1]);
  upk2(dA1, f[2], f[3]);
  reorder(f, x);
  st.store(args.params + part * slab, pk2(f[0], f[1]), pk2(f[2], f[3]));
  if (!last) {
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (cell_t < kTile && cell_d + j < a.D) {
        float* out = args.lanes + (part * 2 * kTile + cell_t) * a.D + cell_d + j;
        out[0] = dskip[j], out[static_cast<int64_t>(kTile) * a.D] = dbias[j];
      }
    return;
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
#pragma unroll
    for (int bit = kPer; bit < 32; bit *= 2) {
      dskip[j] += __shfl_xor_sync(0xffffffffu, dskip[j], bit);
      dbias[j] += __shfl_xor_sync(0xffffffffu, dbias[j], bit);
    }
    if (cell_t == 0 && cell_d + j < a.D) {
      args.channels[part * 2 * a.D + cell_d + j] = dskip[j];
      args.channels[(part * 2 + 1) * a.D + cell_d + j] = dbias[j];
    }
  }
}

// dB and dC [B, T, N] from the blocks' parts, of all tokens or of a piece of every segment;
// zeros behind the last token.
template <typename E, bool PIECE>
__global__ void __launch_bounds__(256) selective_pairs_kernel(SelectiveBwdArgs args) {
  const SelectiveArgs& a = args.f;
  const int64_t rows =
      PIECE ? static_cast<int64_t>(a.segments) * args.tiles_per_piece * kTile : a.T;
  const int64_t wide = 2 * static_cast<int64_t>(a.N), all = a.B * rows * wide;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  wait_for_previous();
  if (i >= all) return;
  const int64_t row = i / wide;
  const int q = static_cast<int>(i % wide), which = q / a.N, s = q % a.N;
  const int b = static_cast<int>(row / rows);
  int64_t t = row % rows;
  if (PIECE) {
    const int each = args.tiles_per_piece * kTile, seg = static_cast<int>(t / each);
    const int64_t end = static_cast<int64_t>(seg + 1) * a.tiles_per_segment * kTile;
    t = t % each + (static_cast<int64_t>(seg) * a.tiles_per_segment +
                    static_cast<int64_t>(args.piece) * args.tiles_per_piece) * kTile;
    if (t >= end || t >= a.T) return;
  }
  float sum = 0.0f;
  if (t < length_of(a.lens, b, a.T))
#pragma unroll 8
    for (int k = 0; k < a.blocks; ++k) sum += args.pairs[k * all + i];
  E* out = static_cast<E*>(which == 0 ? args.dB : args.dC);
  out[(static_cast<int64_t>(b) * a.T + t) * a.N + s] = store_from_float<E>(sum);
}

// dA, dskip and ddt_bias from the parts of sequences and segments.
__global__ void __launch_bounds__(256) selective_params_kernel(SelectiveBwdArgs args) {
  const SelectiveArgs& a = args.f;
  const int64_t slab = static_cast<int64_t>(a.D) * a.N;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  wait_for_previous();
  if (i >= slab + 2 * a.D) return;
  const bool matrix = i < slab;
  const float* from = matrix ? args.params + i : args.channels + (i - slab);
  const int64_t step = matrix ? slab : 2 * a.D, parts = static_cast<int64_t>(a.B) * a.segments;
  float sum = 0.0f;
#pragma unroll 8
  for (int64_t k = 0; k < parts; ++k) sum += from[k * step];
  const int64_t d = i - slab;
  if (matrix)
    args.dA[i] = sum;
  else if (d < a.D ? args.dskip != nullptr : args.ddt_bias != nullptr)
    (d < a.D ? args.dskip : args.ddt_bias - a.D)[d] = sum;
}

template <typename E, int L, bool ALIGNED>
cudaError_t bwd_of(const SelectiveBwdArgs& args, cudaStream_t st) {
  const SelectiveArgs& a = args.f;
  const int64_t blocks = static_cast<int64_t>(a.B) * a.blocks * a.segments;
  cudaError_t e;
  if constexpr (L <= kSegmentLanes)
    if (a.segments > 1) {
      e = launch(selective_bwd_state_kernel<E, L, ALIGNED>, blocks, kThreads,
                 sizeof(BwdStateShared<E, L, ALIGNED>), st, args);
      if (e == cudaSuccess) e = launch_carry(a, args.dh_out, true, st);
      if (e != cudaSuccess) return e;
    }
  SelectiveBwdArgs now = args;
  const int64_t rows = args.pieces == 1 ? a.T
                                        : static_cast<int64_t>(a.segments) * args.tiles_per_piece *
                                              kTile;
  const int64_t pairs = a.B * rows * 2 * a.N;
  for (now.piece = args.pieces - 1; now.piece >= 0; --now.piece) {
    e = launch(selective_bwd_kernel<E, L, ALIGNED>, blocks, kThreads,
               sizeof(BwdShared<E, L, ALIGNED>), st, now);
    if (e == cudaSuccess && pairs > 0)
      e = launch(args.pieces == 1 ? selective_pairs_kernel<E, false>
                                  : selective_pairs_kernel<E, true>,
                 (pairs - 1) / 256 + 1, 256, 0, st, now);
    if (e != cudaSuccess) return e;
  }
  const int64_t params = static_cast<int64_t>(a.D) * (a.N + 2);
  return launch(selective_params_kernel, (params - 1) / 256 + 1, 256, 0, st, args);
}
template <typename E, int L>
cudaError_t bwd(const SelectiveBwdArgs& args, cudaStream_t st) {
  return words<E>(args.f, {args.dy, args.du, args.ddt, args.dz}) ? bwd_of<E, L, true>(args, st)
                                                                : bwd_of<E, L, false>(args, st);
}

constexpr size_t kPairBytes = size_t{512} << 20;  // of dB's and dC's parts, or the marks' if more

// Segments, pieces and the floats of the workspace's parts.
struct Plan {
  int segments, tiles_per_segment, pieces, tiles_per_piece;
  size_t pairs, params, channels, carry, sums, lanes;
};
Plan plan(int B, int T, int D, int N) {
  Plan p{};
  p.segments = selective_segments(B, T, D, N, &p.tiles_per_segment);
  const size_t blocks = selective_blocks(D, N), pair = 2 * static_cast<size_t>(N), tokens = T;
  const size_t marks = static_cast<size_t>(B) * ((tokens + kTile - 1) / kTile) * D * N;
  const size_t most = std::max(kPairBytes / sizeof(float), marks);
  p.pairs = blocks * B * tokens * pair;
  p.pieces = 1, p.tiles_per_piece = p.tiles_per_segment;
  if (selective_lanes(N) > 4 && p.pairs > most) {
    const size_t pieces = std::min<size_t>((p.pairs - 1) / most + 1, p.tiles_per_segment);
    p.tiles_per_piece = static_cast<int>((p.tiles_per_segment - 1) / pieces + 1);
    p.pieces = (p.tiles_per_segment - 1) / p.tiles_per_piece + 1;
  }
  const size_t bs = static_cast<size_t>(B) * p.segments;
  if (p.pieces > 1) p.pairs = blocks * bs * p.tiles_per_piece * kTile * pair;
  p.params = bs * D * N, p.channels = bs * 2 * D;
  p.carry = p.segments > 1 || p.pieces > 1 ? bs * D * N : 0, p.sums = p.segments > 1 ? bs * D : 0;
  p.lanes = p.pieces > 1 ? bs * 2 * kTile * D : 0;
  // (each a multiple of four floats, so that the next starts at 16 bytes)
  for (size_t* n : {&p.pairs, &p.params, &p.channels, &p.carry, &p.sums}) *n = (*n + 3) / 4 * 4;
  return p;
}

}  // namespace

size_t selective_scan_bwd_workspace_bytes(int B, int T, int D, int N) {
  if (B <= 0 || T < 0 || D <= 0 || N <= 0) return 0;
  const Plan p = plan(B, T, D, N);
  return sizeof(float) * (p.pairs + p.params + p.channels + p.carry + p.sums + p.lanes);
}

cudaError_t selective_scan_bwd_launch(SelectiveBwdArgs args, void* workspace, cudaStream_t st) {
  SelectiveArgs& a = args.f;
  if (a.D == 0) {
    const size_t all = static_cast<size_t>(a.B) * a.T * a.N * (a.dtype == SANATAN_F32 ? 4 : 2);
    cudaError_t e = cudaMemsetAsync(args.dB, 0, all, st);
    return e == cudaSuccess ? cudaMemsetAsync(args.dC, 0, all, st) : e;
  }
  if (a.B == 0) {
    const size_t row = static_cast<size_t>(a.D) * sizeof(float);
    cudaError_t e = cudaMemsetAsync(args.dA, 0, row * a.N, st);
    if (e == cudaSuccess && args.dskip != nullptr) e = cudaMemsetAsync(args.dskip, 0, row, st);
    if (e == cudaSuccess && args.ddt_bias != nullptr)
      e = cudaMemsetAsync(args.ddt_bias, 0, row, st);
    return e;
  }
  a.blocks = selective_blocks(a.D, a.N);
  const Plan p = plan(a.B, a.T, a.D, a.N);
  a.segments = p.segments, a.tiles_per_segment = p.tiles_per_segment;
  args.pieces = p.pieces, args.tiles_per_piece = p.tiles_per_piece;
  args.pairs = static_cast<float*>(workspace);
  args.params = args.pairs + p.pairs;
  args.channels = args.params + p.params;
  a.carry = args.channels + p.channels;
  a.sums = a.carry + p.carry;
  args.lanes = a.sums + p.sums;
  a.vec = state_words(a.N, {a.A, args.marks, args.dh_out, args.dh0, args.pairs});
  if (a.dtype == SANATAN_F32) SANATAN_SELECTIVE_DISPATCH(bwd, float, args)
  SANATAN_SELECTIVE_DISPATCH(bwd, __nv_bfloat16, args)
}

}  // namespace sanatan
