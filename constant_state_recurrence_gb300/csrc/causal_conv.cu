// Short causal convolution, per channel of [B, T, D] with K taps (1 .. 8):
//   c_t = bias + sum_k w_k x_{t-K+1+k},   y = c  or  c / (1 + exp(-c)),
// where x_i for i < 0 is the state (the K - 1 inputs before the first token) or zero, its
// gradients, with dc = dy or dy (sg + c sg (1 - sg)), sg = 1 / (1 + exp(-c)),
//   dx_i = sum_j w_{K-1-j} dc_{i+j},   dw_k = sum_t dc_t x_{t-K+1+k},   dbias = sum_t dc_t,
// and the single-token step on the state.  Products and sums are float32.
//
// Bound: bytes (two tensors forward, three backward).  A thread has V neighbouring
// channels of a run of tokens and keeps the last K - 1 inputs in registers, so that a value is
// loaded once but for K - 1 tokens before a run (and, backward, behind it).  Backward, the
// forward's sum is formed again; the thread walks its run once, with the K unfinished dx in
// registers: dc_t goes into each, and dx_{t-K+1} is then done.  The weights' gradients stay in
// registers over all runs of a thread; blocks leave partial sums, and a second kernel adds
// them in a fixed order (no atomics: the same call gives the same bits).
#include <algorithm>
#include <initializer_list>

#include "pdl.cuh"
#include "sanatan_internal.h"
#include "vec_io.cuh"

namespace sanatan {
namespace {

constexpr int kThreads = 128;
constexpr int kRun = 16;        // tokens of a thread, forward
constexpr int kAhead = 8;       // tokens whose loads are under way together
constexpr int kRunBwd = 32;
constexpr int kLanes = 32, kRows = 8;  // backward block: channels x runs
constexpr int kParts = kConvParts;

__device__ __forceinline__ float sigmoid(float c) { return __fdividef(1.0f, 1.0f + __expf(-c)); }

__device__ __forceinline__ int length_of(const int64_t* lens, int b, int T) {
  if (lens == nullptr) return T;
  const int64_t n = lens[b];
  return n < 0 ? 0 : (n > T ? T : static_cast<int>(n));
}

// A sequence's inputs: token i in [-(K-1), n) of V channels from c.
template <typename E, int V>
struct Inputs {
  const E* x;        // token 0
  const float* s;    // the state's first row, or null
  int64_t ld;
  int K, D;
  __device__ __forceinline__ void at(int i, float (&f)[V]) const {
    if (i >= 0) {
      Vec<E, V> v;
      v.load(x + i * ld);
      v.get(f);
    } else if (s != nullptr) {
      Vec<float, V> v;
      v.load(s + static_cast<int64_t>(K - 1 + i) * D);
      v.get(f);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = 0.0f;
    }
  }
};

// Weights of V channels from c: w [D, K], the K taps last of KM (the first KM - K: zeros).
template <int KM, int V>
__device__ __forceinline__ void load_weights(const float* w, int c, int K, float (&f)[KM][V]) {
  const int pad = KM - K;
#pragma unroll
  for (int k = 0; k < KM; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j)
      f[k][j] = k >= pad ? w[static_cast<int64_t>(c + j) * K + k - pad] : 0.0f;
}

// c_t of the window (win: the KM - 1 inputs before, x the token's own).  Taps before the
// first are left out, not multiplied by zero: what they would reach need not be finite.
template <int KM, int V>
__device__ __forceinline__ void convolve(const float (&w)[KM][V], const float (&win)[KM - 1][V],
                                         const float (&x)[V], const float (&bias)[V], int K,
                                         float (&c)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) c[j] = fmaf(w[KM - 1][j], x[j], bias[j]);
#pragma unroll
  for (int k = 0; k < KM - 1; ++k)
    if (KM <= 4 || k >= KM - K)
#pragma unroll
      for (int j = 0; j < V; ++j) c[j] = fmaf(w[k][j], win[k][j], c[j]);
}

template <int N, int V>
__device__ __forceinline__ void push(float (&win)[N][V], const float (&x)[V]) {
#pragma unroll
  for (int k = 0; k + 1 < N; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) win[k][j] = win[k + 1][j];
#pragma unroll
  for (int j = 0; j < V; ++j) win[N - 1][j] = x[j];
}

template <typename E, int KM, int V>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a) {
  const int vecs = a.D / V, K = a.K, pad = KM - K;
  const int64_t runs = static_cast<int64_t>(a.B) * a.runs;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = item / vecs;  // a run, or, behind all of them, a sequence's state
  if (row >= runs + (a.s_out != nullptr ? a.B : 0)) return;
  const int c = static_cast<int>(item % vecs) * V;
  const bool state = row >= runs;
  const int b = static_cast<int>(state ? row - runs : row / a.runs);
  wait_for_previous();
  const int n = length_of(a.lens, b, a.T);
  const E* x0 = static_cast<const E*>(a.x) + static_cast<int64_t>(b) * a.T * a.ldx + c;
  const float* s0 =
      a.s0 == nullptr ? nullptr : a.s0 + static_cast<int64_t>(b) * (K - 1) * a.D + c;
  const Inputs<E, V> in{x0, s0, a.ldx, K, a.D};
  if (state) {
    float* out = a.s_out + static_cast<int64_t>(b) * (K - 1) * a.D + c;
    for (int k = 0; k < K - 1; ++k) {
      float f[V];
      in.at(n - (K - 1) + k, f);
      Vec<float, V> v;
      v.put(f);
      v.store(out + static_cast<int64_t>(k) * a.D);
    }
    return;
  }
  const int t0 = static_cast<int>(row % a.runs) * kRun, end = min(t0 + kRun, a.T);
  E* y = static_cast<E*>(a.y) + (static_cast<int64_t>(b) * a.T + t0) * a.D + c;
  float w[KM][V], bias[V], win[KM - 1][V];
  if (t0 < n) {
    load_weights<KM, V>(a.w, c, K, w);
#pragma unroll
    for (int j = 0; j < V; ++j) bias[j] = a.bias != nullptr ? a.bias[c + j] : 0.0f;
#pragma unroll
    for (int k = 0; k < KM - 1; ++k) {
      if (k >= pad) {
        in.at(t0 - (KM - 1) + k, win[k]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) win[k][j] = 0.0f;
      }
    }
  }
  for (int t = t0; t < end; t += kAhead) {
    Vec<E, V> raw[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (t + i < end && t + i < n) raw[i].load(x0 + (t + i) * a.ldx);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t + i >= end) break;
      float f[V];
      if (t + i < n) {
        float x[V];
        raw[i].get(x);
        convolve<KM, V>(w, win, x, bias, K, f);
        push(win, x);
        if (a.act == SANATAN_ACT_SILU)
#pragma unroll
          for (int j = 0; j < V; ++j) f[j] = __fdividef(f[j], 1.0f + __expf(-f[j]));
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = 0.0f;
      }
      Vec<E, V> o;
      o.put(f);
      o.store(y);
      y += a.D;
    }
  }
}

template <typename E, int KM, int V>
__global__ void __launch_bounds__(kLanes* kRows) conv_bwd_kernel(ConvBwdArgs a) {
  __shared__ float sums[kRows][V][kLanes + 1];
  const int lane = threadIdx.x % kLanes, ty = threadIdx.x / kLanes;
  const int K = a.K, pad = KM - K;
  const int c = (blockIdx.x * kLanes + lane) * V;
  const bool there = c < a.D;
  float w[KM][V], bias[V], dw[KM][V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    db[j] = 0.0f;
#pragma unroll
    for (int k = 0; k < KM; ++k) dw[k][j] = 0.0f;
  }
  wait_for_previous();
  if (there) {
    load_weights<KM, V>(a.w, c, K, w);
#pragma unroll
    for (int j = 0; j < V; ++j) bias[j] = a.bias != nullptr ? a.bias[c + j] : 0.0f;
  }
  const int64_t runs = there ? static_cast<int64_t>(a.B) * a.runs : 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.y) * kRows + ty; row < runs;
       row += static_cast<int64_t>(gridDim.y) * kRows) {
    const int b = static_cast<int>(row / a.runs);
    const int n = length_of(a.lens, b, a.T);
    const int t0 = static_cast<int>(row % a.runs) * kRunBwd, end = min(t0 + kRunBwd, a.T);
    const E* x0 = static_cast<const E*>(a.x) + static_cast<int64_t>(b) * a.T * a.ldx + c;
    const int64_t at = static_cast<int64_t>(b) * a.T * a.D + c;
    const E* dy = static_cast<const E*>(a.dy) + at;
    E* dx = static_cast<E*>(a.dx) + at;
    const int64_t state = static_cast<int64_t>(b) * (K - 1) * a.D + c;
    const Inputs<E, V> in{x0, a.s0 == nullptr ? nullptr : a.s0 + state, a.ldx, K, a.D};
    float win[KM - 1][V], open[KM][V];  // open[k]: dx of token t - (KM - 1) + k so far
#pragma unroll
    for (int k = 0; k < KM; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) open[k][j] = 0.0f;
#pragma unroll
    for (int k = 0; k < KM - 1; ++k) {
      if (k >= pad && t0 < n) {
        in.at(t0 - (KM - 1) + k, win[k]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) win[k][j] = 0.0f;
      }
    }
    // dx is done for tokens from first on: the state's too in the first run
    const int first = t0 == 0 ? -(K - 1) : t0;
    constexpr int kStep = 4;
    for (int t1 = t0; t1 < end + K - 1; t1 += kStep) {
      Vec<E, V> rx[kStep], rd[kStep];
#pragma unroll
      for (int i = 0; i < kStep; ++i)
        if (t1 + i < n && t1 + i < end + K - 1) {
          rx[i].load(x0 + (t1 + i) * a.ldx);
          rd[i].load(dy + static_cast<int64_t>(t1 + i) * a.D);
        }
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int t = t1 + i;
        if (t >= end + K - 1) break;
        if (t < n) {
          float x[V], d[V];
          rx[i].get(x);
          rd[i].get(d);
          if (a.act == SANATAN_ACT_SILU) {
            float f[V];
            convolve<KM, V>(w, win, x, bias, K, f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const float sg = sigmoid(f[j]);
              d[j] *= fmaf(f[j] * sg, 1.0f - sg, sg);
            }
          }
#pragma unroll
          for (int k = 0; k < KM; ++k)
            if (KM <= 4 || k >= pad)
#pragma unroll
              for (int j = 0; j < V; ++j) open[k][j] = fmaf(w[k][j], d[j], open[k][j]);
          if (t < end) {  // (the tokens behind the run are another thread's)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              db[j] += d[j];
              dw[KM - 1][j] = fmaf(d[j], x[j], dw[KM - 1][j]);
#pragma unroll
              for (int k = 0; k < KM - 1; ++k)
                if (KM <= 4 || k >= pad) dw[k][j] = fmaf(d[j], win[k][j], dw[k][j]);
            }
          }
          push(win, x);
        }
        // dx of token o is done
        const int o = t - (K - 1);
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = KM <= 4 ? open[0][j] : 0.0f;
        if (KM > 4)
#pragma unroll
          for (int k = 0; k < KM; ++k)
            if (k == pad)
#pragma unroll
              for (int j = 0; j < V; ++j) f[j] = open[k][j];
        if (o >= first && o < end) {
          const int k = o - (n - (K - 1));  // the state behind the last token holds it
          if (a.ds_out != nullptr && k >= 0 && k < K - 1) {
            Vec<float, V> v;
            float g[V];
            v.load(a.ds_out + state + static_cast<int64_t>(k) * a.D);
            v.get(g);
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] += g[j];
          }
          if (o >= 0) {
            Vec<E, V> v;
            v.put(f);
            v.store(dx + static_cast<int64_t>(o) * a.D);
          } else if (a.ds0 != nullptr) {
            Vec<float, V> v;
            v.put(f);
            v.store(a.ds0 + state + static_cast<int64_t>(K - 1 + o) * a.D);
          }
        }
        const float zero[V] = {};
        push(open, zero);
      }
    }
  }
  if (a.parts == nullptr) return;
  // The block's runs together, tap by tap: part [K + 1][D], the bias last.
  float* part = a.parts + static_cast<int64_t>(blockIdx.y) * (K + 1) * a.D;
#pragma unroll
  for (int k = 0; k <= KM; ++k) {
    if (k < pad) continue;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) sums[ty][j][lane] = k < KM ? dw[k < KM ? k : 0][j] : db[j];
    __syncthreads();
    // (V * kLanes channels, of which each thread adds up some)
    for (int i = threadIdx.x; i < V * kLanes; i += kLanes * kRows) {
      const int j = i % V, l = i / V;
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) s += sums[r][j][l];
      const int ch = (blockIdx.x * kLanes + l) * V + j;
      if (ch < a.D) part[static_cast<int64_t>(k - pad) * a.D + ch] = s;
    }
  }
}

// dw [D, K] and dbias [D] from n parts [K + 1][D].
__global__ void __launch_bounds__(256) conv_parts_kernel(const float* parts, int n, int D, int K,
                                                         float* dw, float* db) {
  __shared__ float all[8][33];
  const int x = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + x;
  const int64_t wide = static_cast<int64_t>(K + 1) * D;
  wait_for_previous();
  float v = 0.0f;
  if (i < wide)
    for (int p = ty; p < n; p += 8) v += parts[p * wide + i];
  all[ty][x] = v;
  __syncthreads();
  if (ty == 0 && i < wide) {
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) s += all[p][x];
    const int64_t k = i / D, c = i % D;
    if (k < K) {
      if (dw != nullptr) dw[c * K + k] = s;
    } else if (db != nullptr) {
      db[c] = s;
    }
  }
}

template <typename E, int KM, int V>
__global__ void __launch_bounds__(kThreads)
    conv_step_kernel(float* state, const E* x, int64_t ldx, const float* w, const float* bias,
                     int act, int N, int D, int K, E* y) {
  const int vecs = D / V, pad = KM - K;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t n = item / vecs;
  if (n >= N) return;
  const int c = static_cast<int>(item % vecs) * V;
  wait_for_previous();
  float* s = state + n * (K - 1) * D + c;
  float wt[KM][V], win[KM - 1][V], b[V], xv[V], f[V];
  Vec<E, V> raw;
  raw.load(x + n * ldx + c);
#pragma unroll
  for (int k = 0; k < KM - 1; ++k) {
    if (k >= pad) {
      Vec<float, V> v;
      v.load(s + static_cast<int64_t>(k - pad) * D);
      v.get(win[k]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) win[k][j] = 0.0f;
    }
  }
  load_weights<KM, V>(w, c, K, wt);
#pragma unroll
  for (int j = 0; j < V; ++j) b[j] = bias != nullptr ? bias[c + j] : 0.0f;
  raw.get(xv);
  convolve<KM, V>(wt, win, xv, b, K, f);
  push(win, xv);
#pragma unroll
  for (int k = 0; k < KM - 1; ++k)
    if (k >= pad) {
      Vec<float, V> v;
      v.put(win[k]);
      v.store(s + static_cast<int64_t>(k - pad) * D);
    }
  if (act == SANATAN_ACT_SILU)
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = __fdividef(f[j], 1.0f + __expf(-f[j]));
  Vec<E, V> o;
  o.put(f);
  o.store(y + n * D + c);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t st,
                   Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

unsigned blocks_of(int64_t items) { return static_cast<unsigned>((items - 1) / kThreads + 1); }

template <typename E, int KM, int V>
cudaError_t fwd(ConvArgs a, cudaStream_t st) {
  a.runs = (a.T + kRun - 1) / kRun;
  const int64_t rows = static_cast<int64_t>(a.B) * a.runs + (a.s_out != nullptr ? a.B : 0);
  if (rows == 0) return cudaSuccess;
  return launch(conv_fwd_kernel<E, KM, V>, dim3(blocks_of(rows * (a.D / V))), kThreads, st, a);
}

template <typename E, int KM, int V>
cudaError_t bwd(ConvBwdArgs a, cudaStream_t st) {
  a.runs = std::max(1, (a.T + kRunBwd - 1) / kRunBwd);  // (the state's gradient without tokens)
  const int n = static_cast<int>(
      std::min<int64_t>(kParts, (static_cast<int64_t>(a.B) * a.runs - 1) / kRows + 1));
  const bool sums = a.dw != nullptr || a.dbias != nullptr;
  if (!sums) a.parts = nullptr;
  const cudaError_t e =
      launch(conv_bwd_kernel<E, KM, V>, dim3((a.D - 1) / (V * kLanes) + 1, n), kLanes * kRows, st,
             a);
  if (e != cudaSuccess || !sums) return e;
  const int64_t wide = static_cast<int64_t>(a.K + 1) * a.D;
  return launch(conv_parts_kernel, dim3(static_cast<unsigned>((wide - 1) / 32 + 1)), 256, st,
                static_cast<const float*>(a.parts), n, a.D, a.K, a.dw, a.dbias);
}

template <typename E, int KM, int V>
cudaError_t step(const ConvArgs& a, cudaStream_t st) {
  return launch(conv_step_kernel<E, KM, V>, dim3(blocks_of(static_cast<int64_t>(a.B) * (a.D / V))),
                kThreads, st, a.s_out, static_cast<const E*>(a.x), a.ldx, a.w, a.bias, a.act, a.B,
                a.D, a.K, static_cast<E*>(a.y));
}

// Whether rows of D values with ldx values between those of x are words of V values at
// every address (states: floats).
template <typename E>
bool words(int V, int D, int64_t ldx, std::initializer_list<const void*> tensors,
           std::initializer_list<const void*> states) {
  if (D % V != 0 || ldx % V != 0) return false;
  for (const void* p : tensors)
    if (!at_bytes(p, V * sizeof(E))) return false;
  for (const void* p : states)
    if (!at_bytes(p, V > 1 ? 16 : 4)) return false;
  return true;
}

}  // namespace

// f<E, KM, V> for the taps and the widest words that every address allows.
#define SANATAN_CONV_DISPATCH(f, E, a, st, vec)                      \
  switch (a.K) {                                                     \
    case 2:                                                          \
      return vec ? f<E, 2, 4>(a, st) : f<E, 2, 1>(a, st);            \
    case 3:                                                          \
      return vec ? f<E, 3, 4>(a, st) : f<E, 3, 1>(a, st);            \
    case 4:                                                          \
      return vec ? f<E, 4, 4>(a, st) : f<E, 4, 1>(a, st);            \
    default:                                                         \
      return vec ? f<E, 8, 4>(a, st) : f<E, 8, 1>(a, st);            \
  }

size_t causal_conv_bwd_workspace_bytes(int B, int T, int D, int K) {
  if (B <= 0 || T < 0 || D <= 0 || K < 1) return 0;
  const int64_t runs = static_cast<int64_t>(B) * std::max(1, T / kRunBwd + (T % kRunBwd != 0));
  const size_t n = static_cast<size_t>(std::min<int64_t>(kParts, (runs - 1) / kRows + 1));
  return sizeof(float) * n * (K + 1) * static_cast<size_t>(D);
}

cudaError_t causal_conv_fwd_launch(const ConvArgs& a, cudaStream_t st) {
  if (a.dtype == SANATAN_F32) {
    const bool vec = words<float>(4, a.D, a.ldx, {a.x, a.y}, {a.s0, a.s_out});
    SANATAN_CONV_DISPATCH(fwd, float, a, st, vec)
  }
  const bool vec = words<__nv_bfloat16>(4, a.D, a.ldx, {a.x, a.y}, {a.s0, a.s_out});
  SANATAN_CONV_DISPATCH(fwd, __nv_bfloat16, a, st, vec)
}

cudaError_t causal_conv_bwd_launch(const ConvBwdArgs& a, cudaStream_t st) {
  if (a.B == 0) {
    const size_t row = static_cast<size_t>(a.D) * sizeof(float);
    cudaError_t e = a.dw != nullptr ? cudaMemsetAsync(a.dw, 0, row * a.K, st) : cudaSuccess;
    if (e == cudaSuccess && a.dbias != nullptr) e = cudaMemsetAsync(a.dbias, 0, row, st);
    return e;
  }
  if (a.dtype == SANATAN_F32) {
    const bool vec = words<float>(4, a.D, a.ldx, {a.x, a.dy, a.dx}, {a.s0, a.ds_out, a.ds0});
    SANATAN_CONV_DISPATCH(bwd, float, a, st, vec)
  }
  const bool vec = words<__nv_bfloat16>(4, a.D, a.ldx, {a.x, a.dy, a.dx}, {a.s0, a.ds_out, a.ds0});
  SANATAN_CONV_DISPATCH(bwd, __nv_bfloat16, a, st, vec)
}

cudaError_t causal_conv_step_launch(const ConvArgs& a, cudaStream_t st) {
  if (a.dtype == SANATAN_F32) {
    const bool vec = words<float>(4, a.D, a.ldx, {a.x, a.y}, {a.s_out});
    SANATAN_CONV_DISPATCH(step, float, a, st, vec)
  }
  const bool vec = words<__nv_bfloat16>(4, a.D, a.ldx, {a.x, a.y}, {a.s_out});
  SANATAN_CONV_DISPATCH(step, __nv_bfloat16, a, st, vec)
}

}  // namespace sanatan
