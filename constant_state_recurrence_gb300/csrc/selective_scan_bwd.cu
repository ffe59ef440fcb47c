// The selective scan's backward (formulas and method: selective_scan.cuh).
//
// A tile's states and decays (sixteen tokens x four states a lane) stay in registers between
// the walk forward from the mark and the walk back, so that a decay is formed once.
#include "selective_scan.cuh"

namespace sanatan {
namespace {

// Shared memory of a block, beside the sums of dB and dC [warp][token][B | C][NP].
template <int L>
struct Shared {
  using G = Geo<L>;
  float4 cells[kTile][G::CB];  // delta, delta, delta u, delta u
  float2 v[kTile][G::CB];      // v, v
  float pairs[kTile][2][G::NP];
  float sums[3][kTile][G::kPitch];  // of dh B, of w A, and y
  float by_warp[kWarps][kTile][2][G::NP];
};

// The walk back alone, from no gradient behind the segment: what its own tokens add to the
// gradient before it, and its sum of delta.
template <typename E, int L>
__global__ void __launch_bounds__(kThreads) selective_bwd_state_kernel(SelectiveBwdArgs args) {
  using G = Geo<L>;
  const SelectiveArgs& a = args.f;
  __shared__ float4 cells[kTile][G::CB];  // delta, delta, v, v
  __shared__ __align__(16) float pairs[kTile][2][G::NP];
  const Place<L> at(a);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, l = lane % L;
  const int mine = warp * G::CW + lane / L;
  const int d0 = at.cb * G::CB, d = d0 + mine;
  const int cell_ch = tid % G::CB, cell_d = d0 + cell_ch;
  const StatePlace st(d, l, a.D, a.N, a.vec);
  wait_for_previous();
  const int n = length_of(a.lens, at.b, a.T);
  const int64_t slab = static_cast<int64_t>(a.D) * a.N;
  float f[kStates];
  st.load(a.A, f);
  const uint64_t A0 = pk2(f[0] * kLog2e, f[1] * kLog2e), A1 = pk2(f[2] * kLog2e, f[3] * kLog2e);
  uint64_t g0 = pk2(0.0f, 0.0f), g1 = g0;
  const bool there = cell_d < a.D;
  const float bias = there && a.dt_bias != nullptr ? a.dt_bias[cell_d] : 0.0f;
  const E* DT = static_cast<const E*>(a.dt);
  const E* Z = static_cast<const E*>(a.z);
  const E* DY = static_cast<const E*>(args.dy);
  const int64_t row0 = static_cast<int64_t>(at.b) * a.T;
  float sum = 0.0f;
  float rdt[G::kItems], rz[G::kItems], rdy[G::kItems];
  PairTile<E, L> pt;
  auto load = [&](int k) {
#pragma unroll
    for (int i = 0; i < G::kItems; ++i) {
      const int cell = tid + i * kThreads, t = k * kTile + cell / G::CB;
      rdt[i] = rz[i] = rdy[i] = 0.0f;
      if (cell < G::kCells && t < n && there) {
        rdt[i] = load_as_float(DT + (row0 + t) * a.D + cell_d);
        rdy[i] = load_as_float(DY + (row0 + t) * a.D + cell_d);
        if (Z != nullptr) rz[i] = load_as_float(Z + (row0 + t) * a.ldz + cell_d);
      }
    }
    pt.load(a, at.b, k * kTile, n);
  };
  const int live = min(at.k1, (n + kTile - 1) / kTile);
  if (at.k0 < live) load(live - 1);
  for (int k = live - 1; k >= at.k0; --k) {
#pragma unroll
    for (int i = 0; i < G::kItems; ++i) {
      const int cell = tid + i * kThreads, t = k * kTile + cell / G::CB;
      float delta = rdt[i] + bias, v = rdy[i];
      if (a.softplus) delta = softplus(delta);
      if (t >= n || !there || cell >= G::kCells) delta = 0.0f;
      if (Z != nullptr) v *= rz[i] * sigmoid(rz[i]);
      sum += delta;
      if (cell < G::kCells) cells[cell / G::CB][cell_ch] = make_float4(delta, delta, v, v);
    }
    pt.put(&pairs[0][0][0]);
    __syncthreads();
    if (k > at.k0) load(k - 1);
#pragma unroll
    for (int t = kTile - 1; t >= 0; --t) {
      const ulonglong2 c = reinterpret_cast<const ulonglong2&>(cells[t][mine]);
      const ulonglong2 Cv = reinterpret_cast<const ulonglong2&>(pairs[t][1][kStates * l]);
      g0 = fmul2(exp2_pair(fmul2(c.x, A0)), ffma2(c.y, Cv.x, g0));
      g1 = fmul2(exp2_pair(fmul2(c.x, A1)), ffma2(c.y, Cv.y, g1));
    }
    __syncthreads();
  }
  st.store(a.carry + (static_cast<int64_t>(at.b) * a.segments + at.seg) * slab, g0, g1);
  float* all = &pairs[0][0][0];
  all[tid] = sum;  // (the tile's readers are done)
  __syncthreads();
  if (tid < G::CB && there) {
    for (int i = tid + G::CB; i < kThreads; i += G::CB) sum += all[i];
    a.sums[(static_cast<int64_t>(at.b) * a.segments + at.seg) * a.D + cell_d] = sum;
  }
}

template <typename E, int L>
__global__ void __launch_bounds__(kThreads, L == 4 || L == 8 ? kSelectiveBwdBlocks : 1)
    selective_bwd_kernel(SelectiveBwdArgs args) {
  using G = Geo<L>;
  const SelectiveArgs& a = args.f;
  extern __shared__ float4 smem4[];
  Shared<L>& sm = *reinterpret_cast<Shared<L>*>(smem4);
  const Place<L> at(a);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, l = lane % L;
  const int mine = warp * G::CW + lane / L;
  const int d0 = at.cb * G::CB, d = d0 + mine;
  const int cell_ch = tid % G::CB, cell_d = d0 + cell_ch;
  const StatePlace st(d, l, a.D, a.N, a.vec);
  wait_for_previous();
  const int n = length_of(a.lens, at.b, a.T);
  const int64_t slab = static_cast<int64_t>(a.D) * a.N;
  const int64_t part = static_cast<int64_t>(at.b) * a.segments + at.seg;
  uint64_t A0, A1, g0, g1, dA0 = pk2(0.0f, 0.0f), dA1 = dA0;
  {
    float f[kStates];
    st.load(a.A, f);
    A0 = pk2(f[0] * kLog2e, f[1] * kLog2e), A1 = pk2(f[2] * kLog2e, f[3] * kLog2e);
    const float* from = a.segments > 1 ? a.carry + part * slab
                        : (args.dh_out != nullptr ? args.dh_out + at.b * slab : nullptr);
    f[0] = f[1] = f[2] = f[3] = 0.0f;
    if (from != nullptr) st.load(from, f);
    g0 = pk2(f[0], f[1]), g1 = pk2(f[2], f[3]);
  }
  const bool there = cell_d < a.D;
  const float bias = there && a.dt_bias != nullptr ? a.dt_bias[cell_d] : 0.0f;
  const float skip = there && a.skip != nullptr ? a.skip[cell_d] : 0.0f;
  const E* U = static_cast<const E*>(a.u);
  const E* DT = static_cast<const E*>(a.dt);
  const E* Z = static_cast<const E*>(a.z);
  const E* DY = static_cast<const E*>(args.dy);
  E* DU = static_cast<E*>(args.du);
  E* DDT = static_cast<E*>(args.ddt);
  E* DZ = static_cast<E*>(args.dz);
  const int64_t row0 = static_cast<int64_t>(at.b) * a.T;
  float dskip = 0.0f, dbias = 0.0f;
  const int live = min(at.k1, (n + kTile - 1) / kTile);

  for (int k = max(at.k0, live); k < at.k1; ++k)  // tiles without a token
    for (int i = 0; i < G::kItems; ++i) {
      const int cell = tid + i * kThreads, t = k * kTile + cell / G::CB;
      if (cell < G::kCells && t < a.T && there) {
        const int64_t o = (row0 + t) * a.D + cell_d;
        DU[o] = DDT[o] = store_from_float<E>(0.0f);
        if (DZ != nullptr) DZ[o] = store_from_float<E>(0.0f);
      }
    }

  float ru[G::kItems], rdt[G::kItems], rz[G::kItems], rdy[G::kItems], rmark[kStates];
  PairTile<E, L> pt;
  auto load = [&](int k) {
    st.load(args.marks + (static_cast<int64_t>(at.b) * at.tiles + k) * slab, rmark);
#pragma unroll
    for (int i = 0; i < G::kItems; ++i) {
      const int cell = tid + i * kThreads, t = k * kTile + cell / G::CB;
      ru[i] = rdt[i] = rz[i] = rdy[i] = 0.0f;
      if (cell < G::kCells && t < n && there) {
        ru[i] = load_as_float(U + (row0 + t) * a.D + cell_d);
        rdt[i] = load_as_float(DT + (row0 + t) * a.D + cell_d);
        rdy[i] = load_as_float(DY + (row0 + t) * a.D + cell_d);
        if (Z != nullptr) rz[i] = load_as_float(Z + (row0 + t) * a.ldz + cell_d);
      }
    }
    pt.load(a, at.b, k * kTile, n);
  };
  if (at.k0 < live) load(live - 1);
  for (int k = live - 1; k >= at.k0; --k) {
    float u[G::kItems], raw[G::kItems], z[G::kItems], dy[G::kItems];
#pragma unroll
    for (int i = 0; i < G::kItems; ++i) {
      const int cell = tid + i * kThreads, t = k * kTile + cell / G::CB;
      u[i] = ru[i], z[i] = rz[i], dy[i] = rdy[i], raw[i] = rdt[i] + bias;
      float delta = a.softplus ? softplus(raw[i]) : raw[i], v = dy[i];
      if (t >= n || !there) delta = 0.0f;
      if (Z != nullptr) v *= z[i] * sigmoid(z[i]);
      if (cell < G::kCells) {
        sm.cells[cell / G::CB][cell_ch] = make_float4(delta, delta, delta * u[i], delta * u[i]);
        sm.v[cell / G::CB][cell_ch] = make_float2(v, v);
      }
    }
    pt.put(&sm.pairs[0][0][0]);
    uint64_t h[kTile + 1][2], decay[kTile][2];
    h[0][0] = pk2(rmark[0], rmark[1]), h[0][1] = pk2(rmark[2], rmark[3]);
    __syncthreads();
    if (k > at.k0) load(k - 1);
#pragma unroll
    for (int g = 0; g < kTile; g += 4) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = g + i;
        const ulonglong2 c = reinterpret_cast<const ulonglong2&>(sm.cells[t][mine]);
        const ulonglong2 Bv = reinterpret_cast<const ulonglong2&>(sm.pairs[t][0][kStates * l]);
        decay[t][0] = exp2_pair(fmul2(c.x, A0)), decay[t][1] = exp2_pair(fmul2(c.x, A1));
        h[t + 1][0] = ffma2(decay[t][0], h[t][0], fmul2(c.y, Bv.x));
        h[t + 1][1] = ffma2(decay[t][1], h[t][1], fmul2(c.y, Bv.y));
        if (Z != nullptr) {
          const ulonglong2 Cv = reinterpret_cast<const ulonglong2&>(sm.pairs[t][1][kStates * l]);
          y[i] = sum2(ffma2(h[t + 1][1], Cv.y, fmul2(h[t + 1][0], Cv.x)));
        }
      }
      if (Z != nullptr) {
        using M = Meet<4, 1, L / 2>;
        M::sum(y, lane);
        if (M::first(lane))
#pragma unroll
          for (int i = 0; i < M::kLeft; ++i) sm.sums[2][g + M::index(lane) + i][mine] = y[i];
      }
    }
#pragma unroll
    for (int g = kTile - 4; g >= 0; g -= 4) {
      float s[8];  // of dh B, then of w A, of four tokens
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const int t = g + i;
        const ulonglong2 c = reinterpret_cast<const ulonglong2&>(sm.cells[t][mine]);
        const uint64_t v = reinterpret_cast<const uint64_t&>(sm.v[t][mine]);
        const ulonglong2 Bv = reinterpret_cast<const ulonglong2&>(sm.pairs[t][0][kStates * l]);
        const ulonglong2 Cv = reinterpret_cast<const ulonglong2&>(sm.pairs[t][1][kStates * l]);
        const uint64_t dh0 = ffma2(v, Cv.x, g0), dh1 = ffma2(v, Cv.y, g1);
        g0 = fmul2(decay[t][0], dh0), g1 = fmul2(decay[t][1], dh1);
        const uint64_t w0 = fmul2(g0, h[t][0]), w1 = fmul2(g1, h[t][1]);
        dA0 = ffma2(w0, c.x, dA0), dA1 = ffma2(w1, c.x, dA1);
        s[i] = sum2(ffma2(dh1, Bv.y, fmul2(dh0, Bv.x)));
        s[4 + i] = sum2(ffma2(w1, A1, fmul2(w0, A0)));
        float p[8];  // the lane's dB, then dC, of its channel
        upk2(fmul2(c.y, dh0), p[0], p[1]);
        upk2(fmul2(c.y, dh1), p[2], p[3]);
        upk2(fmul2(v, h[t + 1][0]), p[4], p[5]);
        upk2(fmul2(v, h[t + 1][1]), p[6], p[7]);
        using M = Meet<8, L, 16>;
        M::sum(p, lane);
        if (M::first(lane))
#pragma unroll
          for (int q = 0; q < M::kLeft; ++q) {
            const int k8 = M::index(lane) + q;
            sm.by_warp[warp][t][k8 / 4][kStates * l + k8 % 4] = p[q];
          }
      }
      using M = Meet<8, 1, L / 2>;
      M::sum(s, lane);
      if (M::first(lane))
#pragma unroll
        for (int q = 0; q < M::kLeft; ++q) {
          const int k8 = M::index(lane) + q;
          sm.sums[k8 / 4][g + k8 % 4][mine] = s[q];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < G::kItems; ++i) {
      const int cell = tid + i * kThreads, tl = cell / G::CB, t = k * kTile + tl;
      if (cell >= G::kCells || t >= a.T || !there) continue;
      const float delta = sm.cells[tl][cell_ch].x, v = sm.v[tl][cell_ch].x;
      const float sB = sm.sums[0][tl][cell_ch], sA = sm.sums[1][tl][cell_ch] * kLn2;
      const float du = fmaf(delta, sB, skip * v);
      float ddt = fmaf(u[i], sB, sA);
      if (a.softplus) ddt *= sigmoid(raw[i]);
      const int64_t o = (row0 + t) * a.D + cell_d;
      const bool real = t < n;
      DU[o] = store_from_float<E>(real ? du : 0.0f);
      DDT[o] = store_from_float<E>(real ? ddt : 0.0f);
      if (Z != nullptr) {
        const float y0 = fmaf(skip, u[i], sm.sums[2][tl][cell_ch]), sg = sigmoid(z[i]);
        const float dz = dy[i] * y0 * fmaf(z[i] * sg, 1.0f - sg, sg);
        DZ[o] = store_from_float<E>(real ? dz : 0.0f);
      }
      if (real) {
        dskip = fmaf(v, u[i], dskip);
        dbias += ddt;
      }
    }
    // dB and dC of the block's channels: [block of channels][b][t][B | C][N]
    float* out = args.pairs + (static_cast<int64_t>(at.cb) * a.B * a.T + row0) * 2 * a.N;
#pragma unroll
    for (int i = 0; i < G::kPairItems; ++i) {
      const int q = tid + i * kThreads, s = q % G::NP, which = q / G::NP % 2;
      const int tl = q / (2 * G::NP), t = k * kTile + tl;
      if (s >= a.N || t >= n) continue;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += sm.by_warp[w][tl][which][s];
      out[(static_cast<int64_t>(t) * 2 + which) * a.N + s] = sum;
    }
    __syncthreads();  // (the next tile's cells take this one's place)
  }
  if (args.dh0 != nullptr && at.seg == 0) st.store(args.dh0 + at.b * slab, g0, g1);
  st.store(args.params + part * slab, dA0, dA1);
  float* all = &sm.sums[0][0][0];
  all[tid] = dskip;
  all[kThreads + tid] = dbias;
  __syncthreads();
  if (tid < G::CB && there) {
    for (int i = tid + G::CB; i < kThreads; i += G::CB) dskip += all[i], dbias += all[kThreads + i];
    args.channels[part * 2 * a.D + cell_d] = dskip;
    args.channels[(part * 2 + 1) * a.D + cell_d] = dbias;
  }
}

// dB and dC [B, T, N] from the blocks' parts; zeros behind the last token.
template <typename E>
__global__ void __launch_bounds__(256) selective_pairs_kernel(SelectiveBwdArgs args) {
  const SelectiveArgs& a = args.f;
  const int64_t wide = 2 * static_cast<int64_t>(a.N), all = static_cast<int64_t>(a.B) * a.T * wide;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  wait_for_previous();
  if (i >= all) return;
  const int64_t row = i / wide;
  const int q = static_cast<int>(i % wide), which = q / a.N, s = q % a.N;
  const int b = static_cast<int>(row / a.T), t = static_cast<int>(row % a.T);
  float sum = 0.0f;
  if (t < length_of(a.lens, b, a.T))
#pragma unroll 8
    for (int k = 0; k < a.blocks; ++k) sum += args.pairs[k * all + i];
  E* out = static_cast<E*>(which == 0 ? args.dB : args.dC);
  out[row * a.N + s] = store_from_float<E>(sum);
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

template <typename E, int L>
cudaError_t bwd(const SelectiveBwdArgs& args, cudaStream_t st) {
  const SelectiveArgs& a = args.f;
  const int64_t blocks = static_cast<int64_t>(a.B) * a.blocks * a.segments;
  cudaError_t e;
  if (a.segments > 1) {
    e = launch(selective_bwd_state_kernel<E, L>, blocks, kThreads, 0, st, args);
    if (e == cudaSuccess) e = launch_carry(a, args.dh_out, true, st);
    if (e != cudaSuccess) return e;
  }
  e = launch(selective_bwd_kernel<E, L>, blocks, kThreads, sizeof(Shared<L>), st, args);
  const int64_t pairs = static_cast<int64_t>(a.B) * a.T * 2 * a.N;
  if (e == cudaSuccess && pairs > 0)
    e = launch(selective_pairs_kernel<E>, (pairs - 1) / 256 + 1, 256, 0, st, args);
  const int64_t params = static_cast<int64_t>(a.D) * (a.N + 2);
  if (e == cudaSuccess)
    e = launch(selective_params_kernel, (params - 1) / 256 + 1, 256, 0, st, args);
  return e;
}

struct Sizes {
  size_t pairs, params, channels, carry, sums;
};
Sizes sizes(int B, int T, int D, int N, int segments) {
  const size_t bs = static_cast<size_t>(B) * segments, several = segments > 1 ? 1 : 0;
  // (each a multiple of four floats, so that the next starts at 16 bytes)
  auto up = [](size_t n) { return (n + 3) / 4 * 4; };
  return {up(static_cast<size_t>(selective_blocks(D, N)) * B * T * 2 * N), up(bs * D * N),
          up(bs * 2 * D), up(several * bs * D * N), up(several * bs * D)};
}

}  // namespace

size_t selective_scan_bwd_workspace_bytes(int B, int T, int D, int N) {
  if (B <= 0 || T < 0 || D <= 0 || N <= 0) return 0;
  int tiles;
  const Sizes s =
      sizes(B, T, D, N, selective_segments(B, T, D, N, kSelectiveBwdBlocks, &tiles));
  return sizeof(float) * (s.pairs + s.params + s.channels + s.carry + s.sums);
}

cudaError_t selective_scan_bwd_launch(SelectiveBwdArgs args, void* workspace, cudaStream_t st) {
  SelectiveArgs& a = args.f;
  if (a.B == 0) {
    const size_t row = static_cast<size_t>(a.D) * sizeof(float);
    cudaError_t e = cudaMemsetAsync(args.dA, 0, row * a.N, st);
    if (e == cudaSuccess && args.dskip != nullptr) e = cudaMemsetAsync(args.dskip, 0, row, st);
    if (e == cudaSuccess && args.ddt_bias != nullptr)
      e = cudaMemsetAsync(args.ddt_bias, 0, row, st);
    return e;
  }
  a.blocks = selective_blocks(a.D, a.N);
  a.segments = selective_segments(a.B, a.T, a.D, a.N, kSelectiveBwdBlocks, &a.tiles_per_segment);
  const Sizes s = sizes(a.B, a.T, a.D, a.N, a.segments);
  args.pairs = static_cast<float*>(workspace);
  args.params = args.pairs + s.pairs;
  args.channels = args.params + s.params;
  a.carry = args.channels + s.channels;
  a.sums = a.carry + s.carry;
  a.vec = state_words(a.N, {a.A, args.marks, args.dh_out, args.dh0, args.pairs});
  if (a.dtype == SANATAN_F32) SANATAN_SELECTIVE_DISPATCH(bwd, float, args)
  SANATAN_SELECTIVE_DISPATCH(bwd, __nv_bfloat16, args)
}

}  // namespace sanatan
