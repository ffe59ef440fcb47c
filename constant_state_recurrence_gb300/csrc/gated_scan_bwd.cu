// Gated linear recurrence: the gradients (the mathematics and the parts shared with
// the forward are in gated_scan.cuh).
#include "gated_scan.cuh"

namespace sanatan {
namespace {

template <typename E, int G, int LANES, bool TMA>
__global__ void __launch_bounds__(kThreads, TMA ? 2 : 1) scan_bwd_kernel(
    const ScanBwdArgs p, const __grid_constant__ Maps maps, int blocks, int cluster_size) {
  constexpr int R = kRunBwd;
  constexpr int kTile = kThreads / LANES * R;  // starts at a mark
  static_assert(kTile % kMark == 0, "tile");
  using Ring = Tiles<E, LANES, TMA, 3, R, kStages>;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(16) Exchange<LANES, true> ex;

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
  Cluster<LANES, true> cluster{ex,   reinterpret_cast<ulonglong2*>(ring + Ring::kBytes),
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
  in.src[2] = static_cast<const E*>(p.dy) + base;
  in.D = D;
  in.len = len;
  in.b = b;
  in.place = place;
  E* dx = static_cast<E*>(p.dx) + static_cast<int64_t>(b) * T * D;
  E* dg = static_cast<E*>(p.dg) + static_cast<int64_t>(b) * T * D;
  const float* marks = p.marks + static_cast<int64_t>(b) * ((T + kMark - 1) / kMark) * D;

  // Tile of step s: rank 0 has the last one, rank 1 the one before it, and so on;
  // -1 past the first.
  auto tile = [&](int s) {
    const int64_t k = tiles - 1 - (static_cast<int64_t>(s) * cluster_size + rank);
    return k < 0 ? -1 : static_cast<int>(k);
  };
  const int run = tid / LANES * R;
  auto begin = [&](int s) { return tile(s) < 0 ? T : tile(s) * kTile; };
  auto token = [&](int s) { return min(begin(s) + run, T); };
  // Warp 0: the gradient that comes into the step's last token from later ones.
  const PairPlace<LANES, TMA> pair(place.c0, at, D);
  uint64_t carry =
      pair.load(p.dh_out == nullptr ? nullptr : p.dh_out + static_cast<int64_t>(b) * D);
  // (in hand before this CTA's first map leaves: the last state may go where it was)
  if (warp == 0) pairs(ex.in[0])[at] = carry;
  if constexpr (TMA) {
    if (tid == kIssuer)
      for (int s = 0; s < kStages; ++s) in.fetch(begin(s), s);
  } else {
    in.prefetch(token(0));
  }
  // Warp 0: the state before the tile of step s, loaded a step ahead.
  auto mark_of = [&](int s) {
    const int k = tile(s);
    return pair.load(k < 0 ? nullptr
                           : marks + static_cast<int64_t>(k) * (kTile / kMark) *
                                         static_cast<int64_t>(D));
  };
  uint64_t next_mark = warp == 0 ? mark_of(0) : 0;

  int slot = 0;
  uint32_t phase = 0;
  for (int s = 0; s < steps; ++s) {
    const int t0 = token(s);
    uint64_t mark = next_mark;
    if (warp == 0) next_mark = mark_of(s + 1);
    if constexpr (TMA) in.wait(slot, phase);
    V4 a[R], keep[R], x[R], dy[R], A, H, P;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      gate<G>(in.get(0, r, slot), a[r], keep[r]);
      x[r] = in.get(1, r, slot);
      dy[r] = in.get(2, r, slot);
    }
    if constexpr (!TMA) in.prefetch(token(s + 1));
    if (t0 + R > len) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        a[r] = select(t0 + r < len, a[r], v4(1.0f));
        if (G == SANATAN_GATE_SIGMOID) keep[r] = select(t0 + r < len, keep[r], v4(0.0f));
        x[r] = select(t0 + r < len, x[r], v4(0.0f));
        dy[r] = select(t0 + r < len, dy[r], v4(0.0f));
      }
    }
    A = v4(1.0f);
    H = P = v4(0.0f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      H = fma(a[r], H, G == SANATAN_GATE_LOG ? x[r] : mul(keep[r], x[r]));
      A = mul(a[r], A);
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) P = mul(a[r], fma(P, v4(1.0f), dy[r]));
    V4 bA, bH, wA, wH, rA, rP, wP;
    warp_scan<LANES, false>(tid, A, H, bA, bH, wA, wH);
    warp_scan<LANES, true>(tid, A, P, rA, rP, wA, wP);
    if ((tid & 31) < LANES) {
      ex.a[warp][lane] = wA;
      ex.h[warp][lane] = wH;
      ex.p[warp][lane] = wP;
    }
    __syncthreads();
    if constexpr (TMA) {  // every warp has read the slot
      if (tid == kIssuer && s + kStages < steps) in.fetch(begin(s + kStages), slot);
    }
    if (warp == 0) {
      uint64_t d = carry;
      if (cluster_size > 1) {
        uint64_t tA = pk2(1.0f, 1.0f), tP = pk2(0.0f, 0.0f);
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
          const uint64_t fa = pairs(ex.a[w])[at];
          tP = ffma2(fa, tP, pairs(ex.p[w])[at]);
          tA = fmul2(fa, tA);
        }
        cluster.share(s, tA, tP);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        pairs(ex.in[w])[at] = mark;
        mark = ffma2(pairs(ex.a[w])[at], mark, pairs(ex.h[w])[at]);
      }
      if (cluster_size > 1) d = cluster.arrive(s, carry);
#pragma unroll
      for (int w = kWarps - 1; w >= 0; --w) {
        pairs(ex.in_p[w])[at] = d;
        d = ffma2(pairs(ex.a[w])[at], d, pairs(ex.p[w])[at]);
      }
      if (cluster_size == 1) carry = d;
    }
    __syncthreads();
    V4 h = fma(bA, ex.in[warp][lane], bH);
    V4 before[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      before[r] = h;
      h = fma(a[r], h, G == SANATAN_GATE_LOG ? x[r] : mul(keep[r], x[r]));
    }
    V4 d = fma(rA, ex.in_p[warp][lane], rP);
    const int64_t last = (static_cast<int64_t>(t0) + R - 1) * D;
    E* to_x = dx + last;
    E* to_g = dg + last;
    const bool whole = t0 + R <= len;
#pragma unroll
    for (int r = R - 1; r >= 0; --r, to_x -= D, to_g -= D) {
      const V4 dh = fma(d, v4(1.0f), dy[r]);
      d = mul(a[r], dh);
      V4 ox = dh, og;
      if (G == SANATAN_GATE_LOG) {
        og = mul(d, before[r]);
      } else {
        ox = mul(dh, keep[r]);
        og = mul(dh, mul(sub(before[r], x[r]), mul(a[r], keep[r])));
      }
      if (whole) {
        place.store(to_x, ox);
        place.store(to_g, og);
      } else if (t0 + r < T) {
        place.store(to_x, select(t0 + r < len, ox, v4(0.0f)));
        place.store(to_g, select(t0 + r < len, og, v4(0.0f)));
      }
    }
    if (++slot == kStages) {
      slot = 0;
      phase ^= 1;
    }
  }
  if (p.dh0 != nullptr && rank == 0 && warp == 0)
    pair.store(p.dh0 + static_cast<int64_t>(b) * D, carry);
  cluster.finish();
}

bool encode_bwd(Maps* m, const ScanBwdArgs& a, int rows, int width) {
  return encode(&m->of[0], a.g, a.dtype, a.B, a.T, a.D, rows, width) &&
         encode(&m->of[1], a.x, a.dtype, a.B, a.T, a.D, rows, width) &&
         encode(&m->of[2], a.dy, a.dtype, a.B, a.T, a.D, rows, width);
}

template <typename E, int G, bool TMA>
cudaError_t bwd_of(const ScanBwdArgs& a, cudaStream_t st, bool* done) {
  return launch_best<scan_bwd_kernel<E, G, 16, TMA>, scan_bwd_kernel<E, G, 8, TMA>, ScanBwdArgs,
                     Tiles<E, 16, TMA, 3, kRunBwd, kStages>,
                     Tiles<E, 8, TMA, 3, kRunBwd, kStages>>(
      a, TMA ? encode_bwd : encode_none<ScanBwdArgs>, st, done);
}
template <typename E, int G>
cudaError_t bwd(const ScanBwdArgs& a, cudaStream_t st) {
  bool done = false;
  // TMA: rows of 16 bytes, from a dy that starts at 16 bytes (a slice of a larger gradient
  // may start at any element, and is read by the element).
  if (a.T > 0 && a.D * sizeof(E) % 16 == 0 && reinterpret_cast<uintptr_t>(a.dy) % 16 == 0) {
    const cudaError_t e = bwd_of<E, G, true>(a, st, &done);
    if (done) return e;
  }
  return bwd_of<E, G, false>(a, st, &done);
}

}  // namespace

int scan_bwd_read_and_clear_error(cudaStream_t st) { return read_and_clear_error(st); }

cudaError_t gated_scan_bwd_launch(const ScanBwdArgs& a, cudaStream_t st) {
  using B16 = __nv_bfloat16;
  if (a.dtype == SANATAN_F32)
    return a.gate == SANATAN_GATE_LOG ? bwd<float, SANATAN_GATE_LOG>(a, st)
                                      : bwd<float, SANATAN_GATE_SIGMOID>(a, st);
  return a.gate == SANATAN_GATE_LOG ? bwd<B16, SANATAN_GATE_LOG>(a, st)
                                    : bwd<B16, SANATAN_GATE_SIGMOID>(a, st);
}

}  // namespace sanatan
