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
// Simplest form: one thread per channel walks the tokens.  The backward
// recomputes h from the forward's marks (the state before every 64th token).
#include "sanatan_internal.h"
#include "sanatan_math.cuh"

namespace sanatan {
namespace {

constexpr int kMark = kScanMark;

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

template <typename E, int G>
__global__ void __launch_bounds__(128) scan_fwd_kernel(const E* __restrict__ x,
                                                       const E* __restrict__ g,
                                                       const int64_t* __restrict__ lens, int T,
                                                       int D, const float* __restrict__ h0,
                                                       E* __restrict__ y, float* __restrict__ h_out,
                                                       float* __restrict__ marks) {
  const int blocks = (D + 127) / 128;
  const int b = blockIdx.x / blocks;
  const int d = (blockIdx.x % blocks) * 128 + threadIdx.x;
  if (d >= D) return;
  const int len = length_of(lens, b, T);
  const int nm = (T + kMark - 1) / kMark;
  float h = h0 != nullptr ? h0[static_cast<int64_t>(b) * D + d] : 0.0f;
  for (int t = 0; t < T; ++t) {
    const int64_t i = (static_cast<int64_t>(b) * T + t) * D + d;
    if (marks != nullptr && t % kMark == 0)
      marks[(static_cast<int64_t>(b) * nm + t / kMark) * D + d] = h;
    if (t < len) {
      float a, keep;
      gate<G>(load_as_float(g + i), a, keep);
      h = fmaf(a, h, keep * load_as_float(x + i));
    }
    y[i] = store_from_float<E>(t < len ? h : 0.0f);
  }
  if (h_out != nullptr) h_out[static_cast<int64_t>(b) * D + d] = h;
}

template <typename E, int G>
__global__ void __launch_bounds__(128) scan_bwd_kernel(
    const E* __restrict__ x, const E* __restrict__ g, const E* __restrict__ dy,
    const int64_t* __restrict__ lens, int T, int D, const float* __restrict__ marks,
    const float* __restrict__ dh_out, E* __restrict__ dx, E* __restrict__ dg,
    float* __restrict__ dh0) {
  const int blocks = (D + 127) / 128;
  const int b = blockIdx.x / blocks;
  const int d = (blockIdx.x % blocks) * 128 + threadIdx.x;
  if (d >= D) return;
  const int len = length_of(lens, b, T);
  const int nm = (T + kMark - 1) / kMark;
  float dh = dh_out != nullptr ? dh_out[static_cast<int64_t>(b) * D + d] : 0.0f;
  float before[kMark];  // h_{t-1} of the stretch
  for (int m = nm - 1; m >= 0; --m) {
    float h = marks[(static_cast<int64_t>(b) * nm + m) * D + d];
    const int t0 = m * kMark, t1 = min(T, t0 + kMark);
    for (int t = t0; t < min(t1, len); ++t) {
      const int64_t i = (static_cast<int64_t>(b) * T + t) * D + d;
      float a, keep;
      gate<G>(load_as_float(g + i), a, keep);
      before[t - t0] = h;
      h = fmaf(a, h, keep * load_as_float(x + i));
    }
    for (int t = t1 - 1; t >= t0; --t) {
      const int64_t i = (static_cast<int64_t>(b) * T + t) * D + d;
      float gx = 0.0f, gg = 0.0f;
      if (t < len) {
        float a, keep;
        gate<G>(load_as_float(g + i), a, keep);
        dh += load_as_float(dy + i);
        const float hp = before[t - t0];
        gx = dh * keep;
        gg = G == SANATAN_GATE_LOG ? dh * (a * hp)
                                   : dh * ((hp - load_as_float(x + i)) * (a * keep));
        dh *= a;
      }
      dx[i] = store_from_float<E>(gx);
      dg[i] = store_from_float<E>(gg);
    }
  }
  if (dh0 != nullptr) dh0[static_cast<int64_t>(b) * D + d] = dh;
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

template <typename E, int G>
cudaError_t fwd(const ScanArgs& a, cudaStream_t st) {
  const int64_t grid = static_cast<int64_t>(a.B) * ((a.D + 127) / 128);
  scan_fwd_kernel<E, G><<<static_cast<unsigned>(grid), 128, 0, st>>>(
      static_cast<const E*>(a.x), static_cast<const E*>(a.g), a.lens, a.T, a.D, a.h0,
      static_cast<E*>(a.y), a.h_out, a.marks);
  return cudaGetLastError();
}

template <typename E, int G>
cudaError_t bwd(const ScanBwdArgs& a, cudaStream_t st) {
  const int64_t grid = static_cast<int64_t>(a.B) * ((a.D + 127) / 128);
  scan_bwd_kernel<E, G><<<static_cast<unsigned>(grid), 128, 0, st>>>(
      static_cast<const E*>(a.x), static_cast<const E*>(a.g), static_cast<const E*>(a.dy), a.lens,
      a.T, a.D, a.marks, a.dh_out, static_cast<E*>(a.dx), static_cast<E*>(a.dg), a.dh0);
  return cudaGetLastError();
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
