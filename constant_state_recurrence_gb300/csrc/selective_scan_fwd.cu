// The selective scan's forward and single-token step (formulas and method: selective_scan.cuh).
#include "selective_scan.cuh"

namespace sanatan {
namespace {

constexpr int kFwdThreads = 2 * kThreads;

template <typename E, int L, bool ALIGNED, bool STATE>
struct FwdShared {
  using G = Geo<L>;
  using Tiles = Stage<E, L, ALIGNED, STATE ? 2 : 3>;  // u, dt, z
  float4 cells[2][kWarps][kTile][G::kRowPitch];       // delta, delta, delta u, delta u
  float pairs[2][kTile][2][1][G::NP];
  float ys[2][kWarps][kTile][G::CW];
  char raw[2][Tiles::kBytes];
};

// STATE: only the segment's result from a zero state, and its sum of delta.
//
// Warps 0 .. 3 walk tile k.  Warps 4 .. 7 work beside them, a warp for the channels of one of
// the first four: they have tile k + 2 copied, form the cells of tile k + 1 and finish the
// outputs of tile k - 1.  All meet once a tile.  (Whole sequences leave an SM ten walking
// warps at the training shape, and each is as slow as its own instructions: walking and the
// rest by the same four warps took 604 us.)
template <typename E, int L, bool ALIGNED, bool STATE>
__global__ void __launch_bounds__(kFwdThreads, L <= 8 ? 3 : 1)
    selective_fwd_kernel(SelectiveArgs a) {
  using G = Geo<L>;
  constexpr int W = G::W;
  using Sm = FwdShared<E, L, ALIGNED, STATE>;
  using Tiles = typename Sm::Tiles;
  extern __shared__ float4 smem4[];
  Sm& sm = *reinterpret_cast<Sm*>(smem4);
  const Place<L> at(a);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 % kWarps;
  const bool walks = threadIdx.x < kThreads;
  const int d0 = at.cb * G::CB, w0 = d0 + warp * G::CW;
  wait_for_previous();
  const int n = length_of(a.lens, at.b, a.T);
  const int64_t slab = static_cast<int64_t>(a.D) * a.N, row0 = static_cast<int64_t>(at.b) * a.T;
  const int64_t part = static_cast<int64_t>(at.b) * a.segments + at.seg;
  const int live = min(at.k1, (n + kTile - 1) / kTile);  // tiles from here on hold no token
  if (walks) {
    const int l = lane / G::CW, mine = lane % G::CW;
    const StatePlace st(w0 + mine, l, a.D, a.N, a.vec);
    uint64_t A0, A1, h0, h1;
    {
      float f[kStates];
      st.load(a.A, f);
      A0 = pk2(f[0] * kLog2e, f[1] * kLog2e), A1 = pk2(f[2] * kLog2e, f[3] * kLog2e);
      const float* from = STATE             ? nullptr
                          : a.segments > 1 ? a.carry + part * slab
                                           : (a.h0 != nullptr ? a.h0 + at.b * slab : nullptr);
      f[0] = f[1] = f[2] = f[3] = 0.0f;
      if (from != nullptr) st.load(from, f);
      h0 = pk2(f[0], f[1]), h1 = pk2(f[2], f[3]);
    }
    if (at.k0 < live) {
      __syncthreads();  // (the first tile's copies)
      __syncthreads();  // (its cells)
    }
    for (int k = at.k0; k < live; ++k) {
      if (!STATE && a.marks != nullptr)
        st.store(a.marks + (static_cast<int64_t>(at.b) * at.tiles + k) * slab, h0, h1);
      const float(*pairs)[2][1][G::NP] = sm.pairs[k & 1];
      const float4(*cells)[G::kRowPitch] = sm.cells[k & 1][warp];
      Decays decays;
#pragma unroll
      for (int g = 0; g < kTile; g += 4) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 c = reinterpret_cast<const ulonglong2&>(cells[g + i][mine]);
          const ulonglong2 Bv =
              reinterpret_cast<const ulonglong2&>(pairs[g + i][0][0][kStates * l]);
          const uint64_t a0 = exp2_pair(fmul2(c.x, A0)), a1 = exp2_pair(fmul2(c.x, A1));
          h0 = ffma2(a0, h0, fmul2(c.y, Bv.x));
          h1 = ffma2(a1, h1, fmul2(c.y, Bv.y));
          decays.add(a0, a1, c.x);
          if (!STATE) {
            const ulonglong2 Cv =
                reinterpret_cast<const ulonglong2&>(pairs[g + i][1][0][kStates * l]);
            v[i] = sum2(ffma2(h1, Cv.y, fmul2(h0, Cv.x)));
          }
        }
        if (!STATE) {
          using M = Meet<4, G::CW, 16>;
          M::sum(v, lane);
          if (M::first(lane))
#pragma unroll
            for (int i = 0; i < M::kLeft; ++i)
              sm.ys[k & 1][warp][g + M::index(lane) + i][mine] = v[i];
        }
      }
      decays.put_right(A0, A1, h0, h1, a.softplus, &cells[0][mine], G::kRowPitch);
      __syncthreads();
    }
    if (STATE)
      st.store(a.carry + part * slab, h0, h1);
    else if (a.h_out != nullptr && at.seg == a.segments - 1)
      st.store(a.h_out + at.b * slab, h0, h1);
    return;
  }
  // The lane's cells: W channels from cell_c of the warp's, token cell_t of a tile.
  constexpr int kPer = G::CW / W, kStep = 32 / kPer;
  const int cell_c = lane % kPer * W, cell_t = lane / kPer, cell_d = w0 + cell_c;
  E* Y = static_cast<E*>(a.y);
  const bool gated = !STATE && a.z != nullptr;
  float bias[W], skip[W], sum[W];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const bool there = cell_d + j < a.D;
    bias[j] = there && a.dt_bias != nullptr ? a.dt_bias[cell_d + j] : 0.0f;
    skip[j] = there && a.skip != nullptr ? a.skip[cell_d + j] : 0.0f;
    sum[j] = 0.0f;
  }
  Tiles tiles;
  if constexpr (STATE)
    tiles.init({a.u, a.dt, a.Bm, nullptr}, {a.D, a.D, a.ldb, 0}, a, row0, n, d0, at.k0, 1);
  else
    tiles.init({a.u, a.dt, a.z, a.Bm, a.Cm}, {a.D, a.D, a.ldz, a.ldb, a.ldc}, a, row0, n, d0,
               at.k0, 1);
  struct Kept {
    float u[W], z[W];
  };
  auto prepare = [&](int k, Kept& kept) {
    Tiles::pairs_to_float(sm.raw[k & 1], a.N, sm.pairs[k & 1]);
    if (!G::kAllLanes && cell_t >= kTile) return;
    float delta[W];
    Tiles::get(sm.raw[k & 1], 0, cell_t, warp * G::CW + cell_c, kept.u);
    Tiles::get(sm.raw[k & 1], 1, cell_t, warp * G::CW + cell_c, delta);
    if (gated) Tiles::get(sm.raw[k & 1], 2, cell_t, warp * G::CW + cell_c, kept.z);
    steps<W>(delta, bias, a.softplus, k * kTile + cell_t < n);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if (STATE) sum[j] += delta[j];
      const float du = delta[j] * kept.u[j];
      sm.cells[k & 1][warp][cell_t][cell_c + j] = make_float4(delta[j], delta[j], du, du);
    }
  };
  auto finish = [&](int k, const Kept& kept) {
    if (!G::kAllLanes && cell_t >= kTile) return;
    const int t = k * kTile + cell_t;
    float y[W];
    Vec<float, W> v;
    v.load(&sm.ys[k & 1][warp][cell_t][cell_c]);
    v.get(y);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      y[j] = fmaf(skip[j], kept.u[j], y[j]);
      if (gated) y[j] *= kept.z[j] * sigmoid(kept.z[j]);
      if (t >= n) y[j] = 0.0f;
    }
    if (t < a.T) store_cells<E, W, ALIGNED>(Y + (row0 + t) * a.D, cell_d, a.D, y);
  };
  Kept before, now, next;  // of tiles k - 1, k, k + 1
  if (at.k0 < live) {
    tiles.begin(sm.raw[at.k0 & 1], at.k0);
    tiles.end(sm.raw[at.k0 & 1]);
    copy_wait<0>();
    __syncthreads();
    if (at.k0 + 1 < live) tiles.begin(sm.raw[(at.k0 + 1) & 1], at.k0 + 1);
    prepare(at.k0, now);
    if (at.k0 + 1 < live) tiles.end(sm.raw[(at.k0 + 1) & 1]);
    copy_wait<0>();
    __syncthreads();
  }
  for (int k = at.k0; k < live; ++k) {
    if (k + 2 < live) tiles.begin(sm.raw[k & 1], k + 2);
    if (k + 1 < live) prepare(k + 1, next);
    if (!STATE && k > at.k0) finish(k - 1, before);
    if (k + 2 < live) tiles.end(sm.raw[k & 1]);
    copy_wait<0>();
    __syncthreads();
    before = now, now = next;
  }
  if constexpr (STATE) {
    // the lanes of a channel, by halves
#pragma unroll
    for (int j = 0; j < W; ++j) {
#pragma unroll
      for (int bit = kPer; bit < 32; bit *= 2) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], bit);
      if (cell_t == 0 && cell_d + j < a.D) a.sums[part * a.D + cell_d + j] = sum[j];
    }
  } else {
    if (at.k0 < live) finish(live - 1, before);
    const float zero[W] = {};
    for (int t = max(at.k0, live) * kTile + cell_t; t < min(at.k1 * kTile, a.T); t += kStep)
      store_cells<E, W, ALIGNED>(Y + (row0 + t) * a.D, cell_d, a.D, zero);  // without a token
  }
}

constexpr int kStepRows = 4;  // sequences of a thread, their states under way together

// One token: four sequences of a channel at a time, L neighbouring lanes a channel.  A lane's
// own sequence of the four is the one whose sum it ends with; it forms delta and the gate of
// that one alone, and the others' come by shuffles.  WORDS: B and C four values at a time.
template <typename E, int L, bool WORDS>
__global__ void __launch_bounds__(kThreads) selective_step_kernel(SelectiveArgs a) {
  using M = Meet<4, 1, L / 2>;
  const int lane = threadIdx.x % 32, l = lane % L;
  const int64_t channels = (static_cast<int64_t>(a.D) + Geo<L>::CB - 1) / Geo<L>::CB;
  const int d = static_cast<int>(blockIdx.x % channels) * Geo<L>::CB +
                static_cast<int>(threadIdx.x) / L;
  const int b0 = static_cast<int>(blockIdx.x / channels) * kStepRows;
  const StatePlace st(d, l, a.D, a.N, a.vec);
  const int64_t slab = static_cast<int64_t>(a.D) * a.N;
  const bool there = d < a.D;
  wait_for_previous();
  float A[kStates], h[kStepRows][kStates];
#pragma unroll
  for (int r = 0; r < kStepRows; ++r)
    if (b0 + r < a.B) st.load(a.h_out + (b0 + r) * slab, h[r]);
  st.load(a.A, A);
  const int own = b0 + M::index(lane);
  const bool real = there && own < a.B;
  float u = 0.0f, delta = 0.0f, z = 0.0f;
  if (real) {
    const int64_t at = static_cast<int64_t>(own) * a.D + d;
    u = load_as_float(static_cast<const E*>(a.u) + at);
    delta = load_as_float(static_cast<const E*>(a.dt) + at);
    if (a.dt_bias != nullptr) delta += a.dt_bias[d];
    if (a.z != nullptr) z = load_as_float(static_cast<const E*>(a.z) + own * a.ldz + d);
  }
  if (a.softplus) {
    float other;
    upk2(softplus_pair(pk2(delta, delta)), delta, other);
  }
  float y[kStepRows];
#pragma unroll
  for (int r = 0; r < kStepRows; ++r) {
    // (index() has the lane's first bit stand for 2, the second for 1)
    const int from = (lane & ~3) | (r >> 1) | (r & 1) << 1;
    const float dr = __shfl_sync(0xffffffffu, delta, from);
    const float du = dr * __shfl_sync(0xffffffffu, u, from), x = dr * kLog2e;
    y[r] = 0.0f;
    if (b0 + r >= a.B) continue;
    float Bv[kStates] = {}, Cv[kStates] = {};
    const E* Bm = static_cast<const E*>(a.Bm) + (b0 + r) * a.ldb + kStates * l;
    const E* Cm = static_cast<const E*>(a.Cm) + (b0 + r) * a.ldc + kStates * l;
    if (WORDS) {
      if (kStates * l < a.N) {
        Vec<E, kStates> v;
        v.load(Bm);
        v.get(Bv);
        v.load(Cm);
        v.get(Cv);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kStates; ++j)
        if (kStates * l + j < a.N) Bv[j] = load_as_float(Bm + j), Cv[j] = load_as_float(Cm + j);
    }
#pragma unroll
    for (int j = 0; j < kStates; ++j) {
      h[r][j] = fmaf(exp2_near(x * A[j]), h[r][j], du * Bv[j]);
      y[r] = fmaf(h[r][j], Cv[j], y[r]);
    }
    st.store(a.h_out + (b0 + r) * slab, pk2(h[r][0], h[r][1]), pk2(h[r][2], h[r][3]));
  }
  M::sum(y, lane);
  if (!M::first(lane) || !real) return;
  float out = y[0];
  if (a.skip != nullptr) out = fmaf(a.skip[d], u, out);
  if (a.z != nullptr) out *= z * sigmoid(z);
  static_cast<E*>(a.y)[static_cast<int64_t>(own) * a.D + d] = store_from_float<E>(out);
}

template <typename E, int L, bool ALIGNED>
cudaError_t fwd_of(const SelectiveArgs& a, cudaStream_t st) {
  const int64_t blocks = static_cast<int64_t>(a.B) * a.blocks * a.segments;
  if constexpr (L <= kSegmentLanes)
    if (a.segments > 1) {
      cudaError_t e =
          launch(selective_fwd_kernel<E, L, ALIGNED, true>, blocks, kFwdThreads,
                 sizeof(FwdShared<E, L, ALIGNED, true>), st, a);
      if (e == cudaSuccess) e = launch_carry(a, a.h0, false, st);
      if (e != cudaSuccess) return e;
    }
  return launch(selective_fwd_kernel<E, L, ALIGNED, false>, blocks, kFwdThreads,
                sizeof(FwdShared<E, L, ALIGNED, false>), st, a);
}
template <typename E, int L>
cudaError_t fwd(const SelectiveArgs& a, cudaStream_t st) {
  return words<E>(a, {a.y}) ? fwd_of<E, L, true>(a, st) : fwd_of<E, L, false>(a, st);
}

template <typename E, int L>
cudaError_t step(const SelectiveArgs& a, cudaStream_t st) {
  const int64_t channels = (a.D - 1) / Geo<L>::CB + 1, rows = (a.B - 1) / kStepRows + 1;
  const bool word = a.N % kStates == 0 && a.ldb % kStates == 0 && a.ldc % kStates == 0 &&
                    at_bytes(a.Bm, kStates * sizeof(E)) && at_bytes(a.Cm, kStates * sizeof(E));
  return word ? launch(selective_step_kernel<E, L, true>, channels * rows, kThreads, 0, st, a)
              : launch(selective_step_kernel<E, L, false>, channels * rows, kThreads, 0, st, a);
}

}  // namespace

// (Fewer than four lanes a channel would take more channels a block, and with them 100 KB of
// shared memory and more: up to sixteen states cost what sixteen do.)
int selective_lanes(int N) {
  int L = 4;
  while (kStates * L < N) L *= 2;
  return L;
}

int selective_blocks(int D, int N) { return (D - 1) / (kThreads / selective_lanes(N)) + 1; }

// Segments of a sequence, and their tiles.  One, where whole sequences make two blocks or more
// an SM (a split walks the tokens twice; training shape, 384 blocks: forward 425 us, backward
// 1390 and, when both walked slower, 1466 whole and 1572 in eight segments); else about six
// blocks an SM (one prompt of 32768 tokens, 48 blocks: 10, 13, 19 and 38 segments forward 852, 747,
// 616 and 622 us, backward 2330, 1847, 1484 and 1471), of four tiles or more.  More than 64
// states: always one.
int selective_segments(int B, int T, int D, int N, int* tiles_per_segment) {
  const int tiles = std::max(1, (T - 1) / kTile + 1);
  const int64_t blocks = static_cast<int64_t>(B) * selective_blocks(D, N);
  int64_t S = 1;
  if (blocks < 2 * kSms && selective_lanes(N) <= kSegmentLanes)
    S = std::min<int64_t>((6 * kSms - 1) / blocks + 1, tiles / 4);
  S = std::max<int64_t>(S, 1);
  *tiles_per_segment = static_cast<int>((tiles - 1) / S + 1);
  return (tiles - 1) / *tiles_per_segment + 1;
}

size_t selective_scan_fwd_workspace_bytes(int B, int T, int D, int N) {
  if (B <= 0 || T <= 0 || D <= 0 || N <= 0) return 0;
  int tiles;
  const int S = selective_segments(B, T, D, N, &tiles);
  return S == 1 ? 0 : sizeof(float) * static_cast<size_t>(B) * S * D * (N + 1);
}

cudaError_t selective_scan_fwd_launch(SelectiveArgs a, void* workspace, cudaStream_t st) {
  a.blocks = selective_blocks(a.D, a.N);
  a.segments = selective_segments(a.B, a.T, a.D, a.N, &a.tiles_per_segment);
  a.carry = static_cast<float*>(workspace);
  if (a.segments > 1) a.sums = a.carry + static_cast<int64_t>(a.B) * a.segments * a.D * a.N;
  a.vec = state_words(a.N, {a.A, a.h0, a.h_out, a.marks, a.carry});
  if (a.dtype == SANATAN_F32) SANATAN_SELECTIVE_DISPATCH(fwd, float, a)
  SANATAN_SELECTIVE_DISPATCH(fwd, __nv_bfloat16, a)
}

cudaError_t selective_scan_step_launch(SelectiveArgs a, cudaStream_t st) {
  a.vec = state_words(a.N, {a.A, a.h_out});
  if (a.dtype == SANATAN_F32) SANATAN_SELECTIVE_DISPATCH(step, float, a)
  SANATAN_SELECTIVE_DISPATCH(step, __nv_bfloat16, a)
}

}  // namespace sanatan
