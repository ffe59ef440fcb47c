// The selective scan's forward and single-token step (formulas and method: selective_scan.cuh).
#include "selective_scan.cuh"

namespace sanatan {
namespace {

// STATE: only the segment's result from a zero state, and its sum of delta.
template <typename E, int L, bool STATE>
__global__ void __launch_bounds__(kThreads) selective_fwd_kernel(SelectiveArgs a) {
  using G = Geo<L>;
  __shared__ float4 cells[kTile][G::CB];  // delta, delta, delta u, delta u
  __shared__ __align__(16) float pairs[kTile][2][G::NP];
  __shared__ float ys[kTile][G::kPitch];
  Place<L> at(a);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, l = lane % L;
  const int mine = warp * G::CW + lane / L;  // the lane's channel of the block
  const int d0 = at.cb * G::CB, d = d0 + mine;
  const int cell_ch = tid % G::CB, cell_d = d0 + cell_ch;  // the thread's in every cell of its
  const StatePlace st(d, l, a.D, a.N, a.vec);
  wait_for_previous();
  const int n = length_of(a.lens, at.b, a.T);
  const int64_t slab = static_cast<int64_t>(a.D) * a.N;
  uint64_t A0, A1, h0, h1;
  {
    float f[kStates];
    st.load(a.A, f);
    A0 = pk2(f[0] * kLog2e, f[1] * kLog2e), A1 = pk2(f[2] * kLog2e, f[3] * kLog2e);
    const float* from = STATE ? nullptr
                        : a.segments > 1
                            ? a.carry + (static_cast<int64_t>(at.b) * a.segments + at.seg) * slab
                            : (a.h0 != nullptr ? a.h0 + at.b * slab : nullptr);
    f[0] = f[1] = f[2] = f[3] = 0.0f;
    if (from != nullptr) st.load(from, f);
    h0 = pk2(f[0], f[1]), h1 = pk2(f[2], f[3]);
  }
  const bool there = cell_d < a.D;
  const float bias = there && a.dt_bias != nullptr ? a.dt_bias[cell_d] : 0.0f;
  const float skip = !STATE && there && a.skip != nullptr ? a.skip[cell_d] : 0.0f;
  const E* U = static_cast<const E*>(a.u);
  const E* DT = static_cast<const E*>(a.dt);
  const E* Z = static_cast<const E*>(a.z);
  E* Y = static_cast<E*>(a.y);
  const int64_t row0 = static_cast<int64_t>(at.b) * a.T;
  float sum = 0.0f;

  float ru[G::kItems], rdt[G::kItems], rz[G::kItems];
  PairTile<E, L> pt;
  auto load = [&](int k) {
#pragma unroll
    for (int i = 0; i < G::kItems; ++i) {
      const int cell = tid + i * kThreads, t = k * kTile + cell / G::CB;
      ru[i] = rdt[i] = rz[i] = 0.0f;
      if (cell < G::kCells && t < n && there) {
        ru[i] = load_as_float(U + (row0 + t) * a.D + cell_d);
        rdt[i] = load_as_float(DT + (row0 + t) * a.D + cell_d);
        if (!STATE && Z != nullptr) rz[i] = load_as_float(Z + (row0 + t) * a.ldz + cell_d);
      }
    }
    pt.load(a, at.b, k * kTile, n);
  };
  const int live = min(at.k1, (n + kTile - 1) / kTile);  // tiles from here on hold no token
  if (at.k0 < live) load(at.k0);
  for (int k = at.k0; k < live; ++k) {
    float u[G::kItems], z[G::kItems];
#pragma unroll
    for (int i = 0; i < G::kItems; ++i) {
      const int cell = tid + i * kThreads, t = k * kTile + cell / G::CB;
      u[i] = ru[i], z[i] = rz[i];
      float delta = rdt[i] + bias;
      if (a.softplus) delta = softplus(delta);
      if (t >= n || !there) delta = 0.0f;  // (a = 1 and no input: the state passes)
      if (STATE) sum += cell < G::kCells ? delta : 0.0f;
      if (cell < G::kCells)
        cells[cell / G::CB][cell_ch] = make_float4(delta, delta, delta * u[i], delta * u[i]);
    }
    pt.put(&pairs[0][0][0]);
    __syncthreads();
    if (k + 1 < live) load(k + 1);
    if (!STATE && a.marks != nullptr)
      st.store(a.marks + (static_cast<int64_t>(at.b) * at.tiles + k) * slab, h0, h1);
#pragma unroll
    for (int g = 0; g < kTile; g += 4) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const ulonglong2 c = reinterpret_cast<const ulonglong2&>(cells[g + i][mine]);
        const ulonglong2 Bv = reinterpret_cast<const ulonglong2&>(pairs[g + i][0][kStates * l]);
        h0 = ffma2(exp2_pair(fmul2(c.x, A0)), h0, fmul2(c.y, Bv.x));
        h1 = ffma2(exp2_pair(fmul2(c.x, A1)), h1, fmul2(c.y, Bv.y));
        if (!STATE) {
          const ulonglong2 Cv = reinterpret_cast<const ulonglong2&>(pairs[g + i][1][kStates * l]);
          v[i] = sum2(ffma2(h1, Cv.y, fmul2(h0, Cv.x)));
        }
      }
      if (!STATE) {
        using M = Meet<4, 1, L / 2>;
        M::sum(v, lane);
        if (M::first(lane))
#pragma unroll
          for (int i = 0; i < M::kLeft; ++i) ys[g + M::index(lane) + i][mine] = v[i];
      }
    }
    __syncthreads();
    if (!STATE)
#pragma unroll
      for (int i = 0; i < G::kItems; ++i) {
        const int cell = tid + i * kThreads, tl = cell / G::CB, t = k * kTile + tl;
        if (cell >= G::kCells || t >= a.T || !there) continue;
        float y = fmaf(skip, u[i], ys[tl][cell_ch]);
        if (Z != nullptr) y *= __fdividef(z[i], 1.0f + __expf(-z[i]));
        Y[(row0 + t) * a.D + cell_d] = store_from_float<E>(t < n ? y : 0.0f);
      }
  }
  if constexpr (STATE) {
    st.store(a.carry + (static_cast<int64_t>(at.b) * a.segments + at.seg) * slab, h0, h1);
    // the threads of a channel, in order
    __syncthreads();
    float* all = &ys[0][0];
    all[tid] = sum;
    __syncthreads();
    if (tid < G::CB && there) {
      for (int i = tid + G::CB; i < kThreads; i += G::CB) sum += all[i];
      a.sums[(static_cast<int64_t>(at.b) * a.segments + at.seg) * a.D + cell_d] = sum;
    }
  } else {
    for (int k = max(at.k0, live); k < at.k1; ++k)  // tiles without a token
      for (int i = 0; i < G::kItems; ++i) {
        const int cell = tid + i * kThreads, t = k * kTile + cell / G::CB;
        if (cell < G::kCells && t < a.T && there)
          Y[(row0 + t) * a.D + cell_d] = store_from_float<E>(0.0f);
      }
    if (a.h_out != nullptr && at.seg == a.segments - 1) st.store(a.h_out + at.b * slab, h0, h1);
  }
}

constexpr int kStepRows = 4;  // sequences of a thread, their states under way together

template <typename E, int L>
__global__ void __launch_bounds__(kThreads) selective_step_kernel(SelectiveArgs a) {
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
  const float bias = there && a.dt_bias != nullptr ? a.dt_bias[d] : 0.0f;
  const float skip = there && a.skip != nullptr ? a.skip[d] : 0.0f;
#pragma unroll
  for (int r = 0; r < kStepRows; ++r) {
    const int b = b0 + r;
    if (b >= a.B) break;
    float u = 0.0f, delta = 0.0f, z = 0.0f;
    if (there) {
      u = load_as_float(static_cast<const E*>(a.u) + static_cast<int64_t>(b) * a.D + d);
      delta = load_as_float(static_cast<const E*>(a.dt) + static_cast<int64_t>(b) * a.D + d) + bias;
      if (a.z != nullptr) z = load_as_float(static_cast<const E*>(a.z) + b * a.ldz + d);
    }
    if (a.softplus) delta = softplus(delta);
    float y = 0.0f, decay[kStates];
    const uint64_t x = pk2(delta * kLog2e, delta * kLog2e);
    upk2(exp2_pair(fmul2(x, pk2(A[0], A[1]))), decay[0], decay[1]);
    upk2(exp2_pair(fmul2(x, pk2(A[2], A[3]))), decay[2], decay[3]);
#pragma unroll
    for (int j = 0; j < kStates; ++j) {
      const int n = kStates * l + j;
      float Bv = 0.0f, Cv = 0.0f;
      if (n < a.N) {
        Bv = load_as_float(static_cast<const E*>(a.Bm) + b * a.ldb + n);
        Cv = load_as_float(static_cast<const E*>(a.Cm) + b * a.ldc + n);
      }
      h[r][j] = fmaf(decay[j], h[r][j], delta * u * Bv);
      y = fmaf(h[r][j], Cv, y);
    }
    st.store(a.h_out + b * slab, pk2(h[r][0], h[r][1]), pk2(h[r][2], h[r][3]));
#pragma unroll
    for (int bit = 1; bit < L; bit *= 2) y += __shfl_xor_sync(0xffffffffu, y, bit);
    y = fmaf(skip, u, y);
    if (a.z != nullptr) y *= __fdividef(z, 1.0f + __expf(-z));
    if (l == 0 && there)
      static_cast<E*>(a.y)[static_cast<int64_t>(b) * a.D + d] = store_from_float<E>(y);
  }
}

template <typename E, int L>
cudaError_t fwd(SelectiveArgs a, cudaStream_t st) {
  const int64_t blocks = static_cast<int64_t>(a.B) * a.blocks * a.segments;
  if (a.segments > 1) {
    cudaError_t e = launch(selective_fwd_kernel<E, L, true>, blocks, kThreads, 0, st, a);
    if (e == cudaSuccess) e = launch_carry(a, a.h0, false, st);
    if (e != cudaSuccess) return e;
  }
  return launch(selective_fwd_kernel<E, L, false>, blocks, kThreads, 0, st, a);
}

template <typename E, int L>
cudaError_t step(const SelectiveArgs& a, cudaStream_t st) {
  const int64_t channels = (a.D - 1) / Geo<L>::CB + 1, rows = (a.B - 1) / kStepRows + 1;
  return launch(selective_step_kernel<E, L>, channels * rows, kThreads, 0, st, a);
}

}  // namespace

int selective_lanes(int N) {
  int L = 1;
  while (kStates * L < N) L *= 2;
  return L;
}

int selective_blocks(int D, int N) { return (D - 1) / (kThreads / selective_lanes(N)) + 1; }

// Segments of a sequence (and their tiles): one, unless the blocks of whole sequences leave
// most SMs without the work that hides a walk's latency.
int selective_segments(int B, int T, int D, int N, int per_sm, int* tiles_per_segment) {
  const int tiles = std::max(1, (T - 1) / kTile + 1);
  const int64_t blocks = static_cast<int64_t>(B) * selective_blocks(D, N);
  const int64_t slots = 152 * per_sm;
  int64_t S = 1;
  if (blocks * 2 < slots) S = std::min<int64_t>((slots * 3 / 2 - 1) / blocks + 1, tiles / 4);
  S = std::max<int64_t>(S, 1);
  *tiles_per_segment = static_cast<int>((tiles - 1) / S + 1);
  return (tiles - 1) / *tiles_per_segment + 1;
}

size_t selective_scan_fwd_workspace_bytes(int B, int T, int D, int N) {
  if (B <= 0 || T <= 0 || D <= 0 || N <= 0) return 0;
  int tiles;
  const int S = selective_segments(B, T, D, N, kSelectiveFwdBlocks, &tiles);
  return S == 1 ? 0 : sizeof(float) * static_cast<size_t>(B) * S * D * (N + 1);
}

cudaError_t selective_scan_fwd_launch(SelectiveArgs a, void* workspace, cudaStream_t st) {
  a.blocks = selective_blocks(a.D, a.N);
  a.segments = selective_segments(a.B, a.T, a.D, a.N, kSelectiveFwdBlocks, &a.tiles_per_segment);
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
