// Short causal convolution, per channel of [B, T, D] with K taps (1 .. 8):
//   c_t = bias + sum_k w_k x_{t-K+1+k},   y = c  or  c / (1 + exp(-c)),
// where x_i for i < 0 is the state (the K - 1 inputs before the first token) or zero, its
// gradients, with dc = dy or dy (sg + c sg (1 - sg)), sg = 1 / (1 + exp(-c)),
//   dx_i = sum_j w_{K-1-j} dc_{i+j},   dw_k = sum_t dc_t x_{t-K+1+k},   dbias = sum_t dc_t,
// and the single-token step on the state.  Products and sums are float32.
//
// Bound: bytes (two tensors forward, three backward).  A thread has V neighbouring
// channels of a run of tokens and keeps the last K - 1 inputs in registers, so that a value is
// loaded once but for K - 1 tokens before a run (and, backward, behind it).  Loads are
// asynchronous copies into a ring of the thread's own in shared memory, twelve tokens ahead:
// registers for as many loads would leave few threads.  Arithmetic is packed, two channels an
// instruction.  Backward, the forward's sum is formed again; the thread walks its run once,
// with the K unfinished dx in registers: dc_t goes into each, and dx_{t-K+1} is then done.
// The weights' gradients stay in registers over all runs of a thread; blocks leave partial
// sums, and a second kernel adds them in a fixed order (no atomics: the same call gives the same
// bits).  B 8 T 4096 D 1536 K 4 bf16, x a half of wider rows, GB300: forward 39 us, 5.1 TB/s
// (0.75 of the measured copy rate), backward 82, 3.7 TB/s (0.54).  With loads into
// registers, four tokens ahead, and weights loaded value by value every sixteen tokens (each such
// load of a warp touches 32 lines) 92 and 153.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "copy_async.cuh"
#include "lanes.cuh"
#include "pdl.cuh"
#include "per_device.h"
#include "sanatan_internal.h"
#include "vec_io.cuh"

namespace sanatan {
namespace {

using namespace lanes;

constexpr int kThreads = 128;
constexpr int kRunShort = 16, kRunLong = 96;  // tokens of a thread, forward: from, to
constexpr int kStep = 4;     // tokens of a group of copies
constexpr int kGroupsFwd = 4, kGroupsBwd = 4;  // groups of a ring
constexpr int kLanes = 32, kRows = 8;  // backward block: channels x runs
constexpr int kParts = kConvParts;

// A sequence's inputs: token i in [-(K-1), n) of V channels.
template <typename E, int V>
struct Inputs {
  const E* x;        // token 0
  const float* s;    // the state's first row, or null
  int64_t ld;
  int K, D;
  __device__ __forceinline__ Lanes<V> at(int i) const {
    float f[V];
    if (i >= 0) {
      Vec<E, V> v;
      v.load(x + i * ld);
      v.get(f);
    } else if (s != nullptr) {
      load_floats(s + static_cast<int64_t>(K - 1 + i) * D, f);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = 0.0f;
    }
    return Lanes<V>::of(f);
  }
};

// A thread's own ring in shared memory: groups of kStep tokens of NT tensors, copied while the
// ones before are worked on (a thread reads only what it has copied: no barrier).
template <typename E, int V, int NT, int GROUPS, int THREADS>
struct Ring {
  static constexpr int kBytes = V * sizeof(E);
  static constexpr int kSlots = GROUPS * kStep * NT;
  static constexpr size_t kShared = static_cast<size_t>(kSlots) * THREADS * kBytes;
  char* base;  // slot 0
  __device__ __forceinline__ explicit Ring(char* shared) : base(shared + threadIdx.x * kBytes) {}
  __device__ __forceinline__ char* slot(int group, int i, int q) const {
    return base + ((group * kStep + i) * NT + q) * (THREADS * kBytes);
  }
  __device__ __forceinline__ void copy(int group, int i, int q, const E* from) const {
    char* to = slot(group, i, q);
    if constexpr (kBytes >= 4) {
      copy_words<kBytes>(to, from);
    } else {
      *reinterpret_cast<E*>(to) = *from;
    }
  }
  __device__ __forceinline__ Lanes<V> get(int group, int i, int q) const {
    Vec<E, V> v;
    float f[V];
    v.load(reinterpret_cast<const E*>(slot(group, i, q)));
    v.get(f);
    return Lanes<V>::of(f);
  }
};

// Weights of V channels from c: w [D, K], the K taps last of KM (the first KM - K: zeros).
template <int KM, int V>
__device__ __forceinline__ void load_weights(const float* w, int c, int K, Lanes<V> (&out)[KM]) {
  const int pad = KM - K;
  float f[V][KM];
  bool words = false;
  if constexpr (KM == 4) {
    words = reinterpret_cast<uintptr_t>(w) % 16 == 0;
    if (words)
#pragma unroll
      for (int j = 0; j < V; ++j) load_floats(w + static_cast<int64_t>(c + j) * KM, f[j]);
  }
  if (!words) {
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int k = 0; k < KM; ++k)
        f[j][k] = k >= pad ? w[static_cast<int64_t>(c + j) * K + k - pad] : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    float g[V];
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = f[j][k];
    out[k] = Lanes<V>::of(g);
  }
}
template <int V>
__device__ __forceinline__ Lanes<V> load_bias(const float* bias, int c) {
  float f[V];
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = bias != nullptr ? bias[c + j] : 0.0f;
  return Lanes<V>::of(f);
}

// c_t of the window (win: the KM - 1 inputs before, x the token's own).  Taps before the
// first are left out, not multiplied by zero: what they would reach need not be finite.
template <int KM, int V>
__device__ __forceinline__ Lanes<V> convolve(const Lanes<V> (&w)[KM], const Lanes<V> (&win)[KM - 1],
                                             const Lanes<V>& x, const Lanes<V>& bias, int K) {
  Lanes<V> c = fma(w[KM - 1], x, bias);
#pragma unroll
  for (int k = 0; k < KM - 1; ++k)
    if (KM <= 4 || k >= KM - K) c = fma(w[k], win[k], c);
  return c;
}

template <int N, int V>
__device__ __forceinline__ void push(Lanes<V> (&win)[N], const Lanes<V>& x) {
#pragma unroll
  for (int k = 0; k + 1 < N; ++k) win[k] = win[k + 1];
  win[N - 1] = x;
}

template <int V>
__device__ __forceinline__ Lanes<V> activate(const Lanes<V>& c, int act) {
  return act == SANATAN_ACT_SILU ? mul(c, sigmoid(c)) : c;
}

template <typename E, int V>
__device__ __forceinline__ void store(E* p, const Lanes<V>& v) {
  float f[V];
  v.get(f);
  Vec<E, V> o;
  o.put(f);
  o.store(p);
}

template <typename E, int KM, int V>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a) {
  extern __shared__ float4 smem4[];
  char* smem = reinterpret_cast<char*>(smem4);
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
      in.at(n - (K - 1) + k).get(f);
      store_floats(out + static_cast<int64_t>(k) * a.D, f);
    }
    return;
  }
  const int t0 = static_cast<int>(row % a.runs) * a.run, end = min(t0 + a.run, a.T);
  const int live = min(end, n);
  E* y = static_cast<E*>(a.y) + (static_cast<int64_t>(b) * a.T + t0) * a.D + c;
  int t = t0;
  if (t < live) {
    const Ring<E, V, 1, kGroupsFwd, kThreads> ring(smem);
    const E* x = x0 + t0 * a.ldx;  // of the next group
    int ahead = t0, into = 0;
    auto begin = [&] {
#pragma unroll
      for (int i = 0; i < kStep; ++i)
        if (ahead + i < live) ring.copy(into, i, 0, x + i * a.ldx);
      copy_commit();
      ahead += kStep, x += kStep * a.ldx, into = into + 1 == kGroupsFwd ? 0 : into + 1;
    };
#pragma unroll
    for (int g = 0; g + 1 < kGroupsFwd; ++g) begin();
    Lanes<V> w[KM], win[KM - 1];
#pragma unroll
    for (int k = 0; k < KM - 1; ++k)
      win[k] = k >= pad ? in.at(t0 - (KM - 1) + k) : Lanes<V>::of(0.0f);
    load_weights<KM, V>(a.w, c, K, w);
    const Lanes<V> bias = load_bias<V>(a.bias, c);
    for (int now = 0; t < live; t += kStep, now = now + 1 == kGroupsFwd ? 0 : now + 1) {
      begin();
      copy_wait<kGroupsFwd - 1>();
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        if (t + i >= live) break;
        const Lanes<V> xv = ring.get(now, i, 0);
        store(y, activate(convolve<KM, V>(w, win, xv, bias, K), a.act));
        push(win, xv);
        y += a.D;
      }
    }
    copy_wait<0>();
    t = live;
  }
  for (; t < end; ++t, y += a.D) store(y, Lanes<V>::of(0.0f));  // behind the last token
}

template <typename E, int KM, int V>
__global__ void __launch_bounds__(kLanes* kRows, KM <= 4 ? 2 : 1) conv_bwd_kernel(ConvBwdArgs a) {
  extern __shared__ float4 smem4[];
  const Ring<E, V, 2, kGroupsBwd, kLanes * kRows> ring(reinterpret_cast<char*>(smem4));
  __shared__ float sums[kRows][V][kLanes + 1];
  const int lane = threadIdx.x % kLanes, ty = threadIdx.x / kLanes;
  const int K = a.K, pad = KM - K;
  const int c = (blockIdx.x * kLanes + lane) * V;
  const bool there = c < a.D;
  const Lanes<V> zero = Lanes<V>::of(0.0f), one = Lanes<V>::of(1.0f);
  Lanes<V> w[KM], dw[KM], bias = zero, db = zero;
#pragma unroll
  for (int k = 0; k < KM; ++k) w[k] = dw[k] = zero;
  wait_for_previous();
  if (there) {
    load_weights<KM, V>(a.w, c, K, w);
    bias = load_bias<V>(a.bias, c);
  }
  const int64_t runs = there ? static_cast<int64_t>(a.B) * a.runs : 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.y) * kRows + ty; row < runs;
       row += static_cast<int64_t>(gridDim.y) * kRows) {
    const int b = static_cast<int>(row / a.runs);
    const int n = length_of(a.lens, b, a.T);
    const int t0 = static_cast<int>(row % a.runs) * a.run, end = min(t0 + a.run, a.T);
    const int64_t at = static_cast<int64_t>(b) * a.T * a.D + c;
    const int64_t state = static_cast<int64_t>(b) * (K - 1) * a.D + c;
    const E* x = static_cast<const E*>(a.x) + static_cast<int64_t>(b) * a.T * a.ldx + c;
    const E* dy = static_cast<const E*>(a.dy) + at;
    E* dx = static_cast<E*>(a.dx) + at;
    const Inputs<E, V> in{x, a.s0 == nullptr ? nullptr : a.s0 + state, a.ldx, K, a.D};
    Lanes<V> win[KM - 1], open[KM];  // open[k]: dx of token t - (KM - 1) + k so far
#pragma unroll
    for (int k = 0; k < KM; ++k) open[k] = zero;
#pragma unroll
    for (int k = 0; k < KM - 1; ++k)
      win[k] = k >= pad && t0 < n ? in.at(t0 - (KM - 1) + k) : zero;
    // dx is done for tokens from first on: the state's too in the first run; the tokens behind
    // the run, up to last, finish its own and are another thread's otherwise.
    const int first = t0 == 0 ? -(K - 1) : t0, last = end + K - 1;
    // The state behind the last token holds the inputs from `held` on.
    const int held = a.ds_out != nullptr ? n - (K - 1) : 1 << 30;
    x += t0 * a.ldx;
    dy += static_cast<int64_t>(t0) * a.D;
    int ahead = t0, into = 0;
    auto begin = [&] {
#pragma unroll
      for (int i = 0; i < kStep; ++i)
        if (ahead + i < n && ahead + i < last) {
          ring.copy(into, i, 0, x + i * a.ldx);
          ring.copy(into, i, 1, dy + static_cast<int64_t>(i) * a.D);
        }
      copy_commit();
      ahead += kStep, x += kStep * a.ldx, dy += static_cast<int64_t>(kStep) * a.D;
      into = into + 1 == kGroupsBwd ? 0 : into + 1;
    };
    // Four tokens from t; INSIDE: all of them the run's, and what they finish is, too.
    auto tokens = [&](int t, int now, auto inside) {
      constexpr bool INSIDE = decltype(inside)::value;
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        if (!INSIDE && t + i >= last) break;
        if (INSIDE || t + i < n) {
          const Lanes<V> xv = ring.get(now, i, 0);
          Lanes<V> d = ring.get(now, i, 1);
          if (a.act == SANATAN_ACT_SILU) {
            const Lanes<V> cv = convolve<KM, V>(w, win, xv, bias, K), sg = sigmoid(cv);
            d = mul(d, fma(mul(cv, sg), sub(one, sg), sg));
          }
#pragma unroll
          for (int k = 0; k < KM; ++k)
            if (KM <= 4 || k >= pad) open[k] = fma(w[k], d, open[k]);
          if (INSIDE || t + i < end) {
            db = add(d, db);
            dw[KM - 1] = fma(d, xv, dw[KM - 1]);
#pragma unroll
            for (int k = 0; k < KM - 1; ++k)
              if (KM <= 4 || k >= pad) dw[k] = fma(d, win[k], dw[k]);
          }
          push(win, xv);
        }
        const int o = t + i - (K - 1);  // its dx is done
        Lanes<V> done = open[0];
        if (KM > 4)
#pragma unroll
          for (int k = 1; k < KM; ++k)
            if (k == pad) done = open[k];
        if (INSIDE) {
          store(dx + static_cast<int64_t>(o) * a.D, done);
        } else if (o >= first && o < end) {
          float f[V];
          if (o >= held && o < n) {
            load_floats(a.ds_out + state + static_cast<int64_t>(o - held) * a.D, f);
            done = add(Lanes<V>::of(f), done);
          }
          if (o >= 0) {
            store(dx + static_cast<int64_t>(o) * a.D, done);
          } else if (a.ds0 != nullptr) {
            done.get(f);
            store_floats(a.ds0 + state + static_cast<int64_t>(K - 1 + o) * a.D, f);
          }
        }
        push(open, zero);
      }
    };
#pragma unroll
    for (int g = 0; g + 1 < kGroupsBwd; ++g) begin();
    int now = 0;
    for (int t = t0; t < last; t += kStep, now = now + 1 == kGroupsBwd ? 0 : now + 1) {
      begin();
      copy_wait<kGroupsBwd - 1>();
      if (t + kStep <= min(end, n) && t - (K - 1) >= max(first, 0) && t + kStep - K < held)
        tokens(t, now, std::true_type{});
      else
        tokens(t, now, std::false_type{});
    }
    copy_wait<0>();
  }
  if (a.parts == nullptr) return;
  // The block's runs together, tap by tap: part [K + 1][D], the bias last.
  float* part = a.parts + static_cast<int64_t>(blockIdx.y) * (K + 1) * a.D;
#pragma unroll
  for (int k = 0; k <= KM; ++k) {
    if (k < pad) continue;
    float f[V];
    (k < KM ? dw[k < KM ? k : 0] : db).get(f);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) sums[ty][j][lane] = f[j];
    __syncthreads();
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
__global__ void __launch_bounds__(1024) conv_parts_kernel(const float* parts, int n, int D, int K,
                                                         float* dw, float* db) {
  __shared__ float all[32][33];
  const int x = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + x;
  const int64_t wide = static_cast<int64_t>(K + 1) * D;
  wait_for_previous();
  float v = 0.0f;
  if (i < wide)
#pragma unroll 4
    for (int p = ty; p < n; p += 32) v += parts[p * wide + i];
  all[ty][x] = v;
  __syncthreads();
  if (ty == 0 && i < wide) {
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < 32; ++p) s += all[p][x];
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
  Lanes<V> wt[KM], win[KM - 1];
  float f[V];
  Vec<E, V> raw;
  raw.load(x + n * ldx + c);
#pragma unroll
  for (int k = 0; k < KM - 1; ++k) {
    win[k] = Lanes<V>::of(0.0f);
    if (k >= pad) {
      load_floats(s + static_cast<int64_t>(k - pad) * D, f);
      win[k] = Lanes<V>::of(f);
    }
  }
  load_weights<KM, V>(w, c, K, wt);
  raw.get(f);
  const Lanes<V> xv = Lanes<V>::of(f), b = load_bias<V>(bias, c);
  store(y + n * D + c, activate(convolve<KM, V>(wt, win, xv, b, K), act));
  push(win, xv);
#pragma unroll
  for (int k = 0; k < KM - 1; ++k)
    if (k >= pad) {
      win[k].get(f);
      store_floats(s + static_cast<int64_t>(k - pad) * D, f);
    }
}

unsigned blocks_of(int64_t items) { return static_cast<unsigned>((items - 1) / kThreads + 1); }

// Forward blocks that the current device holds at once; asked once a device (again after a
// failure).
template <typename E, int KM, int V>
cudaError_t held(int* blocks) {
  static PerDevice<int> known;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return known.get(dev, blocks, [](int* out) {
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
        &n, conv_fwd_kernel<E, KM, V>, kThreads, Ring<E, V, 1, kGroupsFwd, kThreads>::kShared);
    *out = kSms * std::max(n, 1);
    return e;
  });
}

template <typename E, int KM, int V>
cudaError_t fwd(ConvArgs a, cudaStream_t st) {
  const int64_t vecs = a.D / V, states = a.s_out != nullptr ? a.B : 0;
  constexpr size_t shared = Ring<E, V, 1, kGroupsFwd, kThreads>::kShared;
  static_assert(shared <= 48 * 1024, "no opt-in");
  int at_once = 0;  // blocks that the device holds
  const cudaError_t e = held<E, KM, V>(&at_once);
  if (e != cudaSuccess) return e;
  // The run length whose rounds of blocks take a thread the fewest tokens, those about a run's
  // start (3 K: what is read twice, weights) among them.  B 8 T 4096 D 1536 bf16, with the call
  // around it: 84 tokens, one round, 45 us; 64, a second round that is not full, 49; 16, five
  // rounds, 64.  B 4 T 2048 D 1536 f32: 28 tokens 22.5, 64 24.6.
  int64_t least = INT64_MAX;
  for (int run = kRunShort; run <= kRunLong; run += kStep) {
    const int64_t items = (static_cast<int64_t>(a.B) * ((a.T + run - 1) / run) + states) * vecs;
    const int64_t rounds = (items - 1) / (static_cast<int64_t>(at_once) * kThreads) + 1;
    const int64_t cost = rounds * (run + 3 * a.K);
    if (cost < least) least = cost, a.run = run;
  }
  a.runs = (a.T + a.run - 1) / a.run;
  const int64_t rows = static_cast<int64_t>(a.B) * a.runs + (a.s_out != nullptr ? a.B : 0);
  if (rows == 0) return cudaSuccess;
  return launch_pdl(conv_fwd_kernel<E, KM, V>, dim3(blocks_of(rows * vecs)), kThreads, shared, st,
                    a);
}

// Blocks of runs (kRows of them a block at a time) and tokens of a run, backward: as many
// blocks as two an SM make, each of which adds up the weights' gradients in registers over its
// runs; and of the run lengths the one that costs a thread the fewest tokens, those that it
// reads twice (K - 1 before a run and behind it) among them.
struct Runs {
  int n, run, runs;
};
Runs runs_of(int B, int T, int D, int K, int V) {
  const int64_t columns = (D - 1) / (V * kLanes) + 1;
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(kParts, 2 * kSms / columns));
  Runs best{1, 16, std::max(1, T / 16 + (T % 16 != 0))};  // (one run: the state's gradient)
  int64_t least = INT64_MAX;
  for (int run = 16; run <= 64; run += 8) {
    const int64_t runs = std::max(1, T / run + (T % run != 0));
    const int64_t rounds = (B * runs - 1) / (blocks * kRows) + 1, cost = rounds * (run + 3 * K);
    if (cost < least) {
      least = cost;
      best = {static_cast<int>(std::min(blocks, (B * runs - 1) / kRows + 1)), run,
              static_cast<int>(runs)};
    }
  }
  return best;
}

template <typename E, int KM, int V>
cudaError_t bwd(ConvBwdArgs a, cudaStream_t st) {
  const Runs r = runs_of(a.B, a.T, a.D, a.K, V);
  a.run = r.run, a.runs = r.runs;
  const int n = r.n;
  const bool sums = a.dw != nullptr || a.dbias != nullptr;
  if (!sums) a.parts = nullptr;
  constexpr size_t shared = Ring<E, V, 2, kGroupsBwd, kLanes * kRows>::kShared;
  if (shared > 40 * 1024) {  // (with the block's own)
    const cudaError_t e =
        cudaFuncSetAttribute(conv_bwd_kernel<E, KM, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(shared));
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((a.D - 1) / (V * kLanes) + 1, n);
  const cudaError_t e =
      launch_pdl(conv_bwd_kernel<E, KM, V>, grid, kLanes * kRows, shared, st, a);
  if (e != cudaSuccess || !sums) return e;
  const int64_t wide = static_cast<int64_t>(a.K + 1) * a.D;
  return launch_pdl(conv_parts_kernel, dim3(static_cast<unsigned>((wide - 1) / 32 + 1)), 1024, 0,
                    st, static_cast<const float*>(a.parts), n, a.D, a.K, a.dw, a.dbias);
}

template <typename E, int KM, int V>
cudaError_t step(const ConvArgs& a, cudaStream_t st) {
  const int64_t items = static_cast<int64_t>(a.B) * (a.D / V);
  return launch_pdl(conv_step_kernel<E, KM, V>, dim3(blocks_of(items)), kThreads, 0, st, a.s_out,
                    static_cast<const E*>(a.x), a.ldx, a.w, a.bias, a.act, a.B, a.D, a.K,
                    static_cast<E*>(a.y));
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
    if (!at_bytes(p, V >= 4 ? 16 : 4 * V)) return false;
  return true;
}

}  // namespace

// f<E, KM, V> for the taps, with V channels a thread where every address allows it.
#define SANATAN_CONV_DISPATCH(f, E, V, a, st, vec)                   \
  switch (a.K) {                                                     \
    case 2:                                                          \
      return vec ? f<E, 2, V>(a, st) : f<E, 2, 1>(a, st);            \
    case 3:                                                          \
      return vec ? f<E, 3, V>(a, st) : f<E, 3, 1>(a, st);            \
    case 4:                                                          \
      return vec ? f<E, 4, V>(a, st) : f<E, 4, 1>(a, st);            \
    default:                                                         \
      return vec ? f<E, 8, 4>(a, st) : f<E, 8, 1>(a, st); \
  }

size_t causal_conv_bwd_workspace_bytes(int B, int T, int D, int K) {
  if (B <= 0 || T < 0 || D <= 0 || K < 1) return 0;
  const int n = std::max(runs_of(B, T, D, K, 1).n, runs_of(B, T, D, K, 4).n);
  return sizeof(float) * static_cast<size_t>(n) * (K + 1) * static_cast<size_t>(D);
}

cudaError_t causal_conv_fwd_launch(const ConvArgs& a, cudaStream_t st) {
  if (a.dtype == SANATAN_F32) {
    const bool vec = words<float>(4, a.D, a.ldx, {a.x, a.y}, {a.s0, a.s_out});
    SANATAN_CONV_DISPATCH(fwd, float, 4, a, st, vec)
  }
  const bool vec = words<__nv_bfloat16>(8, a.D, a.ldx, {a.x, a.y}, {a.s0, a.s_out});
  SANATAN_CONV_DISPATCH(fwd, __nv_bfloat16, 8, a, st, vec)
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
    SANATAN_CONV_DISPATCH(bwd, float, 4, a, st, vec)
  }
  const bool vec = words<__nv_bfloat16>(4, a.D, a.ldx, {a.x, a.dy, a.dx}, {a.s0, a.ds_out, a.ds0});
  SANATAN_CONV_DISPATCH(bwd, __nv_bfloat16, 4, a, st, vec)
}

cudaError_t causal_conv_step_launch(const ConvArgs& a, cudaStream_t st) {
  if (a.dtype == SANATAN_F32) {
    const bool vec = words<float>(4, a.D, a.ldx, {a.x, a.y}, {a.s_out});
    SANATAN_CONV_DISPATCH(step, float, 4, a, st, vec)
  }
  const bool vec = words<__nv_bfloat16>(4, a.D, a.ldx, {a.x, a.y}, {a.s_out});
  SANATAN_CONV_DISPATCH(step, __nv_bfloat16, 4, a, st, vec)
}

}  // namespace sanatan
