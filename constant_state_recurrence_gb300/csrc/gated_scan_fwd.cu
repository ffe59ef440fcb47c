// Gated linear recurrence: the forward scan and the single-token step (the
// mathematics and the parts shared with the backward are in gated_scan.cuh).
#include "gated_scan.cuh"

namespace sanatan {
namespace {

template <typename E, int G, int LANES, bool TMA>
__global__ void __launch_bounds__(kThreads, TMA ? 2 : 1) scan_fwd_kernel(
    const ScanArgs p, const __grid_constant__ Maps maps, int blocks, int cluster_size) {
  constexpr int R = kRunFwd<E>;
  constexpr int kTile = kThreads / LANES * R;
  using Ring = Tiles<E, LANES, TMA, 2, R, kStages>;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(16) Exchange<LANES, false> ex;

  const int rank = static_cast<int>(blockIdx.x % cluster_size);
  const int unit = static_cast<int>(blockIdx.x / cluster_size);
  const int b = unit / blocks;
  const int tid = threadIdx.x, lane = tid % LANES, warp = tid >> 5;
  const int T = p.T, D = p.D;
  const Place<LANES, TMA> place{(unit % blocks) * 4 * LANES, lane, D};
  const int tiles = (T + kTile - 1) / kTile;
  const int steps = (tiles + cluster_size - 1) / cluster_size;

  // What touches no tensor comes before the wait for the kernel before.
  const int at = tid % (2 * LANES);
  Cluster<LANES, false> cluster{ex,   reinterpret_cast<ulonglong2*>(ring + Ring::kBytes),
                                 rank, cluster_size, steps, at};
  Ring in;
  in.ring = ring;
  in.full = ex.ring;
  in.maps = &maps;
  in.dead = &cluster.dead;
  in.start(tid);
  cluster.start();
  wait_for_previous();

  const int len = length_of(p.lens, b, T);
  const int64_t base = static_cast<int64_t>(b) * T * D + place.channel(0);
  in.src[0] = static_cast<const E*>(p.g) + base;
  in.src[1] = static_cast<const E*>(p.x) + base;
  in.D = D;
  in.len = len;
  in.b = b;
  in.place = place;
  E* y = static_cast<E*>(p.y) + static_cast<int64_t>(b) * T * D;

  // First token of the CTA's tile in step s, and of the thread's run; T or more past
  // the last one (T is at most 2^30, so a few tiles more fit an int).
  const int run = tid / LANES * R;
  auto begin = [&](int s) { return (s * cluster_size + rank) * kTile; };
  auto token = [&](int s) { return begin(s) + run; };
  // Warp 0: the state before the step's first tile.
  const PairPlace<LANES, TMA> pair(place.c0, at, D);
  uint64_t carry = pair.load(p.h0 == nullptr ? nullptr : p.h0 + static_cast<int64_t>(b) * D);
  // (in hand before this CTA's first map leaves: the last state may go where it was)
  if (warp == 0) pairs(ex.in[0])[at] = carry;
  if constexpr (TMA) {
    if (tid == kIssuer)
      for (int s = 0; s < kStages; ++s) in.fetch(begin(s), s);
  } else {
    in.prefetch(token(0));
  }

  int slot = 0;
  uint32_t phase = 0;
  for (int s = 0; s < steps; ++s) {
    const int t0 = token(s);
    if constexpr (TMA) in.wait(slot, phase);
    // The run's decays and inputs, and its map.
    V4 a[R], u[R], A, H;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      V4 keep;
      gate<G>(in.get(0, r, slot), a[r], keep);
      u[r] = in.get(1, r, slot);
      if (G == SANATAN_GATE_SIGMOID) u[r] = mul(keep, u[r]);
    }
    if constexpr (!TMA) in.prefetch(token(s + 1));
    if (t0 + R > len) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        a[r] = select(t0 + r < len, a[r], v4(1.0f));
        u[r] = select(t0 + r < len, u[r], v4(0.0f));
      }
    }
    A = a[0];
    H = u[0];
#pragma unroll
    for (int r = 1; r < R; ++r) {
      H = fma(a[r], H, u[r]);
      A = mul(a[r], A);
    }
    // The runs of the warp, the warps of the CTA, the CTAs of the cluster.
    V4 bA, bH, wA, wH;
    warp_scan<LANES, false>(tid, A, H, bA, bH, wA, wH);
    if ((tid & 31) < LANES) {
      ex.a[warp][lane] = wA;
      ex.h[warp][lane] = wH;
    }
    __syncthreads();
    if constexpr (TMA) {  // every warp has read the slot
      if (tid == kIssuer && s + kStages < steps) in.fetch(begin(s + kStages), slot);
    }
    if (warp == 0) {
      uint64_t h = carry;
      if (cluster_size > 1) {
        uint64_t tA = pk2(1.0f, 1.0f), tH = pk2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const uint64_t fa = pairs(ex.a[w])[at];
          tH = ffma2(fa, tH, pairs(ex.h[w])[at]);
          tA = fmul2(fa, tA);
        }
        cluster.share(s, tA, tH);
        h = cluster.arrive(s, carry);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        pairs(ex.in[w])[at] = h;
        h = ffma2(pairs(ex.a[w])[at], h, pairs(ex.h[w])[at]);
      }
      if (cluster_size == 1) carry = h;
    }
    __syncthreads();
    V4 h = fma(bA, ex.in[warp][lane], bH);
    if (p.marks != nullptr && t0 % kMark == 0 && t0 < T)
      place.store(p.marks + (static_cast<int64_t>(b) * ((T + kMark - 1) / kMark) + t0 / kMark) * D,
                  h);
    E* row = y + static_cast<int64_t>(t0) * D;
    if (t0 + R <= len) {
#pragma unroll
      for (int r = 0; r < R; ++r, row += D) {
        h = fma(a[r], h, u[r]);
        place.store(row, h);
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r, row += D) {
        h = fma(a[r], h, u[r]);
        if (t0 + r < T) place.store(row, select(t0 + r < len, h, v4(0.0f)));
      }
    }
    if (++slot == kStages) {
      slot = 0;
      phase ^= 1;
    }
  }
  if (p.h_out != nullptr && rank == 0 && warp == 0)
    pair.store(p.h_out + static_cast<int64_t>(b) * D, carry);
  cluster.finish();
}

// One token: four elements a thread (the tensors are dense, so rows do not matter) for
// the first 4 * quads, the others by a thread each.
template <typename E, int G>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(float* __restrict__ h,
                                                             const E* __restrict__ x,
                                                             const E* __restrict__ g, int64_t n,
                                                             int64_t quads, E* __restrict__ y) {
  using Q = Quad<E>;
  using QF = Quad<float>;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  wait_for_previous();
  V4 gv, xv, hv;
  const int64_t last = 4 * quads + (i - quads);
  if (i < quads) {
    hv = QF::get(reinterpret_cast<const QF::type*>(h)[i]);
    gv = Q::get(reinterpret_cast<const typename Q::type*>(g)[i]);
    xv = Q::get(reinterpret_cast<const typename Q::type*>(x)[i]);
  } else if (last < n) {
    hv = v4(h[last]);
    gv = v4(load_as_float(g + last));
    xv = v4(load_as_float(x + last));
  } else {
    return;
  }
  V4 a, keep;
  gate<G>(gv, a, keep);
  hv = fma(a, hv, G == SANATAN_GATE_SIGMOID ? mul(keep, xv) : xv);
  if (i < quads) {
    reinterpret_cast<QF::type*>(h)[i] = QF::put(hv);
    reinterpret_cast<typename Q::type*>(y)[i] = Q::put(hv);
  } else {
    float f[4];
    get(hv, f);
    h[last] = f[0];
    y[last] = store_from_float<E>(f[0]);
  }
}

bool encode_fwd(Maps* m, const ScanArgs& a, int rows, int width) {
  return encode(&m->of[0], a.g, a.dtype, a.B, a.T, a.D, rows, width) &&
         encode(&m->of[1], a.x, a.dtype, a.B, a.T, a.D, rows, width);
}

template <typename E, int G, bool TMA>
cudaError_t fwd_of(const ScanArgs& a, cudaStream_t st, bool* done) {
  return launch_best<scan_fwd_kernel<E, G, 16, TMA>, scan_fwd_kernel<E, G, 8, TMA>, ScanArgs,
                     Tiles<E, 16, TMA, 2, kRunFwd<E>, kStages>,
                     Tiles<E, 8, TMA, 2, kRunFwd<E>, kStages>>(
      a, TMA ? encode_fwd : encode_none<ScanArgs>, st, done);
}
template <typename E, int G>
cudaError_t fwd(const ScanArgs& a, cudaStream_t st) {
  bool done = false;
  if (a.T > 0 && a.D * sizeof(E) % 16 == 0) {
    const cudaError_t e = fwd_of<E, G, true>(a, st, &done);
    if (done) return e;
  }
  return fwd_of<E, G, false>(a, st, &done);
}

template <typename E, int G>
cudaError_t step(float* h, const void* x, const void* g, int64_t n, void* y, cudaStream_t st) {
  // (the state of one sequence of a batch may start at any float)
  const int64_t quads = reinterpret_cast<uintptr_t>(h) % 16 == 0 ? n / 4 : 0;
  const int64_t threads = quads + (n - 4 * quads);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, scan_step_kernel<E, G>, h, static_cast<const E*>(x),
                            static_cast<const E*>(g), n, quads, static_cast<E*>(y));
}

}  // namespace

int scan_fwd_read_and_clear_error(cudaStream_t st) { return read_and_clear_error(st); }

cudaError_t gated_scan_fwd_launch(const ScanArgs& a, cudaStream_t st) {
  using B16 = __nv_bfloat16;
  if (a.dtype == SANATAN_F32)
    return a.gate == SANATAN_GATE_LOG ? fwd<float, SANATAN_GATE_LOG>(a, st)
                                      : fwd<float, SANATAN_GATE_SIGMOID>(a, st);
  return a.gate == SANATAN_GATE_LOG ? fwd<B16, SANATAN_GATE_LOG>(a, st)
                                    : fwd<B16, SANATAN_GATE_SIGMOID>(a, st);
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
