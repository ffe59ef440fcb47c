// Layer norm of rows of D values, with the residual sum before it:
//   s = x + r (rounded to the type: what is stored is what is normalised),
//   mean = sum(s) / D,  var = sum((s - mean)^2) / D,  rstd = 1 / sqrt(var + eps),
//   y = (s - mean) rstd w + b,
// and its gradients, with g = dy w and n = (s - mean) rstd:
//   dx = rstd (g - sum(g) / D - n sum(g n) / D) + ds,  dw = sum_rows dy n,  db = sum_rows dy.
// Means, variances and all sums are float32; the variance is that of the differences from the
// mean, which are in registers, so a mean far from zero costs it nothing.
//
// Bound: bytes.  Forward: a warp holds a row of up to 1024 values in registers, in loads of 16
// bytes, a block one of up to 1024 loads; every value is read once.  32768 x 768 bf16 with the
// residual, GB300: 35 us, 5.8 TB/s (0.85 of the measured copy rate); with weights and bias loaded
// value by value and 112 registers a thread 60.  Backward: a group of threads holds one load of
// a row each, takes two rows at a time, so that the sums over a row cost one barrier for two, and
// keeps its columns' dw and db in registers over all rows of the block; the rows of its next two
// turns are copied to shared memory meanwhile.  47 us with the sums, 4.3 TB/s (0.63), 41 without.
// (At first, without copies ahead: four rows at a time and 12 warps an SM 57, two and 24 warps
// 62.)  Blocks leave partial sums, which a second kernel adds in a fixed order (no atomics: the
// same call gives the same bits).  Rows longer than that are read again from L2 instead of held.
#include <algorithm>
#include <initializer_list>

#include "copy_async.cuh"
#include "pdl.cuh"
#include "sanatan_internal.h"
#include "vec_io.cuh"

namespace sanatan {
namespace {

constexpr int kRowWarps = 4;      // rows of a block, a warp a row
constexpr int kMostThreads = 1024;
constexpr int kRows = 2;          // of a group at a time, backward
constexpr int kGroupThreads = 288;  // threads of a backward block that holds several groups
constexpr int kParts = kNormParts;
constexpr int kAhead = 2;         // turns of a group whose rows are under way, backward
template <int R>
constexpr int kRing = (kAhead + 1) * R * 3;  // 16-byte places of a thread
constexpr int kLoopThreads = 512;

template <typename E>
constexpr int kVec = 16 / sizeof(E);

// The i-th V values of thread t of G in a row: one aligned word, or (rows that start at any
// element) values G apart, so that neighbouring threads read neighbours.
template <typename E, bool ALIGNED>
struct Part;
template <typename E>
struct Part<E, true> {
  static constexpr int V = kVec<E>;
  Vec<E, V> v;
  __device__ __forceinline__ static int col(int t, int G, int i, int j) {
    return (i * G + t) * V + j;
  }
  __device__ __forceinline__ void load(const E* row, int t, int G, int i, int D) {
    const int c = col(t, G, i, 0);
    if (c < D)
      v.load(row + c);
    else
      v.raw = {};
  }
  __device__ __forceinline__ void get(float (&f)[V]) const { v.get(f); }
  __device__ __forceinline__ static void store(E* row, int t, int G, int i, int D,
                                               const float (&f)[V]) {
    const int c = col(t, G, i, 0);
    Vec<E, V> o;
    o.put(f);
    if (c < D) o.store(row + c);
  }
};
template <typename E>
struct Part<E, false> {
  static constexpr int V = kVec<E>;
  E e[V];
  __device__ __forceinline__ static int col(int t, int G, int i, int j) {
    return t + (i * V + j) * G;
  }
  __device__ __forceinline__ void load(const E* row, int t, int G, int i, int D) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = col(t, G, i, j);
      e[j] = c < D ? row[c] : store_from_float<E>(0.0f);
    }
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = load_as_float(e + j);
  }
  __device__ __forceinline__ static void store(E* row, int t, int G, int i, int D,
                                               const float (&f)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = col(t, G, i, j);
      if (c < D) row[c] = store_from_float<E>(f[j]);
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The sum over a block's threads, for all of them.  red [32]: not in use by another sum.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_sum(lane < static_cast<int>(blockDim.x) / 32 ? red[lane] : 0.0f);
}

// s = x + r as it is stored.
template <typename E>
__device__ __forceinline__ float rounded_sum(float x, float r) {
  const E s = store_from_float<E>(x + r);
  return load_as_float(&s);
}

// Weight and bias of a column (null: 1 and 0), and of a part's.
__device__ __forceinline__ float weight_of(const float* w, int c) { return w ? w[c] : 1.0f; }
__device__ __forceinline__ float bias_of(const float* b, int c) { return b ? b[c] : 0.0f; }
template <typename E, bool ALIGNED>
__device__ __forceinline__ void param_of(const float* p, float none, int t, int G, int i, int D,
                                         float (&f)[kVec<E>]) {
  using P = Part<E, ALIGNED>;
#pragma unroll
  for (int j = 0; j < P::V; ++j) f[j] = none;
  if (p == nullptr) return;
  if (ALIGNED) {
    if (P::col(t, G, i, 0) < D) load_floats(p + P::col(t, G, i, 0), f);
  } else {
#pragma unroll
    for (int j = 0; j < P::V; ++j)
      if (P::col(t, G, i, j) < D) f[j] = p[P::col(t, G, i, j)];
  }
}

// A row in registers: WARP: of a warp, NV parts a lane; else of the block.
template <typename E, int NV, bool ALIGNED, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRowWarps : kMostThreads,
                                  WARP ? (NV * kVec<E> <= 24 ? 8 : 6) : 1)
    norm_fwd_kernel(NormArgs a) {
  using P = Part<E, ALIGNED>;
  constexpr int V = P::V;
  __shared__ float red[2][32];
  const int G = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int64_t row =
      WARP ? static_cast<int64_t>(blockIdx.x) * kRowWarps + threadIdx.x / 32 : blockIdx.x;
  const int D = a.D;
  wait_for_previous();
  if (row >= a.rows) return;  // (WARP: the whole warp; otherwise never)
  P p[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) p[i].load(static_cast<const E*>(a.x) + row * D, t, G, i, D);
  float s[NV][V];
  if (a.residual != nullptr) {
    P q[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      q[i].load(static_cast<const E*>(a.residual) + row * D, t, G, i, D);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V];
      p[i].get(s[i]);
      q[i].get(f);
#pragma unroll
      for (int j = 0; j < V; ++j) s[i][j] = rounded_sum<E>(s[i][j], f[j]);
      if (a.sum != nullptr) P::store(static_cast<E*>(a.sum) + row * D, t, G, i, D, s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i].get(s[i]);
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) m += s[i][j];  // (zeros past the end)
  const float inv = 1.0f / D;
  const float mean = (WARP ? warp_sum(m) : block_sum(m, red[0])) * inv;
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[i][j] -= mean;
      q = fmaf(P::col(t, G, i, j) < D ? s[i][j] : 0.0f, s[i][j], q);
    }
  const float var = (WARP ? warp_sum(q) : block_sum(q, red[1])) * inv;
  const float rstd = 1.0f / sqrtf(var + a.eps);
  if (a.stats != nullptr && t == 0) {
    a.stats[2 * row] = mean;
    a.stats[2 * row + 1] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[V], f[V];
    param_of<E, ALIGNED>(a.weight, 1.0f, t, G, i, D, w);
    param_of<E, ALIGNED>(a.bias, 0.0f, t, G, i, D, f);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = fmaf(s[i][j] * rstd, w[j], f[j]);
    P::store(static_cast<E*>(a.y) + row * D, t, G, i, D, f);
  }
}

// A row too long for registers, read three times (twice from L2).
template <typename E>
__global__ void __launch_bounds__(kLoopThreads) norm_fwd_long_kernel(NormArgs a) {
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x;
  const int D = a.D;
  wait_for_previous();
  const E* x = static_cast<const E*>(a.x) + row * D;
  const E* r = a.residual == nullptr ? nullptr : static_cast<const E*>(a.residual) + row * D;
  E* sum = a.sum == nullptr ? nullptr : static_cast<E*>(a.sum) + row * D;
  E* y = static_cast<E*>(a.y) + row * D;
  // (sum may be the residual: what a thread reads again is then the sum already)
  const bool summed = r != nullptr && sum != nullptr;
  auto value = [&](int c, bool first) {
    if (summed && !first) return load_as_float(sum + c);
    const float v = load_as_float(x + c);
    return r == nullptr ? v : rounded_sum<E>(v, load_as_float(r + c));
  };
  float m = 0.0f;
  for (int c = threadIdx.x; c < D; c += kLoopThreads) {
    const float v = value(c, true);
    if (summed) sum[c] = store_from_float<E>(v);
    m += v;
  }
  const float inv = 1.0f / D;
  const float mean = block_sum(m, red[0]) * inv;
  float q = 0.0f;
  for (int c = threadIdx.x; c < D; c += kLoopThreads) {
    const float d = value(c, false) - mean;
    q = fmaf(d, d, q);
  }
  const float rstd = 1.0f / sqrtf(block_sum(q, red[1]) * inv + a.eps);
  if (a.stats != nullptr && threadIdx.x == 0) {
    a.stats[2 * row] = mean;
    a.stats[2 * row + 1] = rstd;
  }
  for (int c = threadIdx.x; c < D; c += kLoopThreads) {
    const float n = (value(c, false) - mean) * rstd;
    y[c] = store_from_float<E>(fmaf(n, weight_of(a.weight, c), bias_of(a.bias, c)));
  }
}

// The sums of N values a lane over the warp: lane l < N has the l-th one's (N a power of two
// up to 32; the values meet while they are halved, 2 N shuffles fewer than one by one).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
#pragma unroll
  for (int n = N / 2, bit = 1; n > 0; n /= 2, bit *= 2) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
  float s = v[0];
#pragma unroll
  for (int bit = N; bit < 32; bit *= 2) s += __shfl_xor_sync(0xffffffffu, s, bit);
  return s;
}
// The index of lane l's sum: its low bits, first halving first.
template <int N>
__device__ __forceinline__ int warp_sums_index(int lane) {
  int k = 0;
#pragma unroll
  for (int n = N / 2, bit = 1; n > 0; n /= 2, bit *= 2) k += (lane & bit) ? n : 0;
  return k;
}

__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Groups of G threads, one load of a row a thread, R rows at a time.  Where rows are words, the
// rows of the next kAhead turns are copied to a ring in shared memory meanwhile, in which each
// thread has places of its own (32768 x 768 bf16: see the head).
template <typename E, bool ALIGNED, int R, int MOST>
__global__ void __launch_bounds__(MOST, MOST == kGroupThreads ? 2 : 1)
    norm_bwd_kernel(NormBwdArgs a, int G, float* parts) {
  using P = Part<E, ALIGNED>;
  constexpr int V = P::V;
  constexpr int N = 2 * R;
  extern __shared__ float4 smem4[];
  // the ring [turn][row][s | dy | ds][thread], then [groups][2][warps of a group][N] sums, then
  // [2 * V][G] columns of the groups before
  const int groups = blockDim.x / G, warps = G / 32;
  const int group = threadIdx.x / G, t = threadIdx.x % G, lane = threadIdx.x % 32;
  float4* ring = smem4 + threadIdx.x;
  float* sums = reinterpret_cast<float*>(smem4 + (ALIGNED ? kRing<R> * blockDim.x : 0));
  float* red = sums + group * (2 * warps * N);
  float* columns = sums + groups * (2 * warps * N);
  const int D = a.D;
  const float inv = 1.0f / D;
  const bool there = P::col(t, G, 0, 0) < D;
  float w[V], dw[V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) dw[j] = db[j] = 0.0f;
  wait_for_previous();
  param_of<E, ALIGNED>(a.weight, 1.0f, t, G, 0, D, w);  // (past the end dy is zero)
  const int mine = warp_sums_index<N>(lane);
  int turn = 0, into = 0, now = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups * R;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * groups + group) * R;
  int64_t ahead = first;
  auto place = [&](int k, int r, int q) { return ring + ((k * R + r) * 3 + q) * blockDim.x; };
  auto copy = [&] {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (there && ahead + r < a.rows) {
        const int64_t at = (ahead + r) * D + P::col(t, G, 0, 0);
        copy_words<16>(place(into, r, 0), static_cast<const E*>(a.s) + at);
        copy_words<16>(place(into, r, 1), static_cast<const E*>(a.dy) + at);
        if (a.ds != nullptr) copy_words<16>(place(into, r, 2), static_cast<const E*>(a.ds) + at);
      }
    copy_commit();
    ahead += step, into = into == kAhead ? 0 : into + 1;
  };
  auto load = [&](P& p, int r, int q, const void* x, int64_t row) {
    if constexpr (ALIGNED) {
      if (there && row < a.rows)
        p.v.load(reinterpret_cast<const E*>(place(now, r, q)));
      else
        p.v.raw = {};
    } else {
      // (a row past the end: zeros, nothing is read)
      p.load(static_cast<const E*>(x) + row * D, t, G, 0, row < a.rows ? D : 0);
    }
  };
  if constexpr (ALIGNED)
#pragma unroll
    for (int k = 0; k < kAhead; ++k) copy();
  for (int64_t row0 = first; row0 < a.rows; row0 += step, turn ^= 1) {
    P s[R], dy[R];
    float mean[R], rstd[R];
    if constexpr (ALIGNED) {
      copy();
      copy_wait<kAhead>();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      load(s[r], r, 0, a.s, row0 + r);
      load(dy[r], r, 1, a.dy, row0 + r);
      mean[r] = row0 + r < a.rows ? a.stats[2 * (row0 + r)] : 0.0f;
      rstd[r] = row0 + r < a.rows ? a.stats[2 * (row0 + r) + 1] : 0.0f;
    }
    float v[N];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float f[V], g[V];
      s[r].get(f);
      dy[r].get(g);
      v[2 * r] = v[2 * r + 1] = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = (f[j] - mean[r]) * rstd[r], gw = g[j] * w[j];
        v[2 * r] += gw;
        v[2 * r + 1] = fmaf(gw, n, v[2 * r + 1]);
        dw[j] = fmaf(g[j], n, dw[j]);
        db[j] += g[j];
      }
    }
    const float sum = warp_sums<N>(v, lane);
    float* half = red + turn * (warps * N);  // (the other half may still be read)
    if (lane < N) half[(t / 32) * N + mine] = sum;
    group_sync(1 + group, G);
    float total[N];
#pragma unroll
    for (int k = 0; k < N; ++k) total[k] = 0.0f;
    for (int k = 0; k < warps; ++k)
#pragma unroll
      for (int q = 0; q < N; ++q) total[q] += half[k * N + q];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r >= a.rows) break;
      float f[V], g[V];
      s[r].get(f);
      dy[r].get(g);
      const float c1 = total[2 * r] * inv, c2 = total[2 * r + 1] * inv;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = (f[j] - mean[r]) * rstd[r];
        f[j] = rstd[r] * (fmaf(g[j], w[j], -c1) - n * c2);
      }
      if (a.ds != nullptr) {
        P ds;
        load(ds, r, 2, a.ds, row0 + r);
        ds.get(g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] += g[j];
      }
      P::store(static_cast<E*>(a.dx) + (row0 + r) * D, t, G, 0, D, f);
    }
    now = now == kAhead ? 0 : now + 1;
  }
  if constexpr (ALIGNED) copy_wait<0>();
  if (parts == nullptr) return;
  // The groups' columns, one group after the other, then the block's part.
  for (int k = 0; k < groups; ++k) {
    if (k == group) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float* cw = columns + j * G + t;
        float* cb = columns + (V + j) * G + t;
        if (k > 0) dw[j] += *cw, db[j] += *cb;
        if (k + 1 < groups) {
          *cw = dw[j], *cb = db[j];
        } else {
          const int c = P::col(t, G, 0, j);
          float* out = parts + static_cast<int64_t>(blockIdx.x) * 2 * D;
          if (c < D) out[c] = dw[j], out[D + c] = db[j];
        }
      }
    }
    __syncthreads();
  }
}

// dx of rows too long for that: sums first, then the row again.
template <typename E>
__global__ void __launch_bounds__(kLoopThreads) norm_bwd_long_kernel(NormBwdArgs a) {
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x;
  const int D = a.D;
  wait_for_previous();
  const E* s = static_cast<const E*>(a.s) + row * D;
  const E* dy = static_cast<const E*>(a.dy) + row * D;
  const E* ds = a.ds == nullptr ? nullptr : static_cast<const E*>(a.ds) + row * D;
  E* dx = static_cast<E*>(a.dx) + row * D;
  const float mean = a.stats[2 * row], rstd = a.stats[2 * row + 1];
  float v1 = 0.0f, v2 = 0.0f;
  for (int c = threadIdx.x; c < D; c += kLoopThreads) {
    const float g = load_as_float(dy + c) * weight_of(a.weight, c);
    v1 += g;
    v2 = fmaf(g, (load_as_float(s + c) - mean) * rstd, v2);
  }
  const float inv = 1.0f / D;
  const float c1 = block_sum(v1, red[0]) * inv, c2 = block_sum(v2, red[1]) * inv;
  for (int c = threadIdx.x; c < D; c += kLoopThreads) {
    const float g = load_as_float(dy + c) * weight_of(a.weight, c);
    float d = rstd * (g - c1 - (load_as_float(s + c) - mean) * rstd * c2);
    if (ds != nullptr) d += load_as_float(ds + c);
    dx[c] = store_from_float<E>(d);
  }
}

// The same rows' dw and db: 32 columns a block, eight rows at a time of its share.
template <typename E>
__global__ void __launch_bounds__(256) norm_columns_kernel(NormBwdArgs a, float* parts) {
  __shared__ float all[2][8][33];
  const int x = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + x, D = a.D;
  wait_for_previous();
  float dw = 0.0f, db = 0.0f;
  if (c < D)
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * 8 + ty; row < a.rows;
         row += static_cast<int64_t>(gridDim.y) * 8) {
      const float g = load_as_float(static_cast<const E*>(a.dy) + row * D + c);
      const float v = load_as_float(static_cast<const E*>(a.s) + row * D + c);
      dw = fmaf(g, (v - a.stats[2 * row]) * a.stats[2 * row + 1], dw);
      db += g;
    }
  all[0][ty][x] = dw;
  all[1][ty][x] = db;
  __syncthreads();
  if (ty < 2 && c < D) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += all[ty][k][x];
    parts[(static_cast<int64_t>(blockIdx.y) * 2 + ty) * D + c] = sum;
  }
}

// dw and db from the blocks' parts [n][2][D].
__global__ void __launch_bounds__(1024) norm_parts_kernel(const float* parts, int n, int D,
                                                          float* dw, float* db) {
  __shared__ float all[32][33];
  const int x = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + x, wide = 2 * static_cast<int64_t>(D);
  wait_for_previous();
  float v = 0.0f;
  if (c < wide)
#pragma unroll 4
    for (int k = ty; k < n; k += 32) v += parts[k * wide + c];
  all[ty][x] = v;
  __syncthreads();
  if (ty == 0 && c < wide) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) sum += all[k][x];
    if (c < D) {
      if (dw != nullptr) dw[c] = sum;
    } else if (db != nullptr) {
      db[c - D] = sum;
    }
  }
}

constexpr int up32(int n) { return (n + 31) / 32 * 32; }

// Shared memory of a backward block of `groups` groups of G threads.
template <typename E, bool ALIGNED, int R>
constexpr size_t bwd_shared(int groups, int G) {
  return sizeof(float) *
             (groups * (2 * (G / 32) * 2 * R) + (groups > 1 ? 2 * kVec<E> * G : 0)) +
         (ALIGNED ? static_cast<size_t>(kRing<R>) * G * groups * 16 : 0);
}

// The limit of shared memory belongs to the function, for all threads and streams of a device:
// it is set to what any width takes, so that two calls at once set the same.
template <typename E, bool ALIGNED, int R, int MOST>
cudaError_t launch_bwd(const NormBwdArgs& a, int n, int groups, int G, float* parts,
                       cudaStream_t st) {
  // (one group of MOST threads, or several: G is at most half of them, groups G all)
  constexpr size_t kOne = bwd_shared<E, ALIGNED, R>(1, MOST);
  constexpr size_t kMost = kOne + sizeof(float) * (R == kRows ? kVec<E> * MOST : 0);
  static_assert(R < kRows || MOST / 32 < 16, "a group has a barrier of its own, of sixteen");
  const auto kernel = norm_bwd_kernel<E, ALIGNED, R, MOST>;
  if (kMost > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMost));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(n), G * groups, bwd_shared<E, ALIGNED, R>(groups, G), st, a, G,
                    parts);
}

template <typename E, bool ALIGNED>
cudaError_t fwd(const NormArgs& a, cudaStream_t st) {
  constexpr int V = kVec<E>;
  const unsigned rows = static_cast<unsigned>(a.rows);
  if (a.D <= 1024) {
    constexpr int kRowThreads = 32 * kRowWarps;
    const dim3 grid((rows - 1) / kRowWarps + 1);
    // 8, 16, 24 or 32 values a lane
    switch ((a.D - 1) / 256) {
      case 0:
        return launch_pdl(norm_fwd_kernel<E, 8 / V, ALIGNED, true>, grid, kRowThreads, 0, st, a);
      case 1:
        return launch_pdl(norm_fwd_kernel<E, 16 / V, ALIGNED, true>, grid, kRowThreads, 0, st, a);
      case 2:
        return launch_pdl(norm_fwd_kernel<E, 24 / V, ALIGNED, true>, grid, kRowThreads, 0, st, a);
      default:
        return launch_pdl(norm_fwd_kernel<E, 32 / V, ALIGNED, true>, grid, kRowThreads, 0, st, a);
    }
  }
  if (a.D <= kMostThreads * V)
    return launch_pdl(norm_fwd_kernel<E, 1, ALIGNED, false>, dim3(rows),
                      up32((a.D - 1) / V + 1), 0, st, a);
  return launch_pdl(norm_fwd_long_kernel<E>, dim3(rows), kLoopThreads, 0, st, a);
}

template <typename E, bool ALIGNED>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t st) {
  constexpr int V = kVec<E>;
  const bool columns = a.dweight != nullptr || a.dbias != nullptr;
  float* parts = columns ? a.parts : nullptr;
  cudaError_t e;
  int n = 0;
  if (a.D <= kMostThreads * V) {
    const int G = up32((a.D - 1) / V + 1);
    const bool several = G <= kGroupThreads;
    const int groups = several ? kGroupThreads / G : 1, R = several ? kRows : 1;
    n = static_cast<int>(std::min<int64_t>(kParts, (a.rows - 1) / (groups * R) + 1));
    e = several ? launch_bwd<E, ALIGNED, kRows, kGroupThreads>(a, n, groups, G, parts, st)
                : launch_bwd<E, ALIGNED, 1, kMostThreads>(a, n, groups, G, parts, st);
  } else {
    e = launch_pdl(norm_bwd_long_kernel<E>, dim3(static_cast<unsigned>(a.rows)), kLoopThreads, 0,
                   st, a);
    if (e == cudaSuccess && columns) {
      n = static_cast<int>(std::min<int64_t>(32, (a.rows - 1) / 8 + 1));
      e = launch_pdl(norm_columns_kernel<E>, dim3((a.D - 1) / 32 + 1, n), 256, 0, st, a, parts);
    }
  }
  if (e != cudaSuccess || !columns) return e;
  return launch_pdl(norm_parts_kernel, dim3(static_cast<unsigned>((2ll * a.D - 1) / 32 + 1)), 1024,
                    0, st, static_cast<const float*>(parts), n, a.D, a.dweight, a.dbias);
}

bool vectors(int D, int dtype, std::initializer_list<const void*> all) {
  if (D % (dtype == SANATAN_F32 ? 4 : 8) != 0) return false;
  for (const void* p : all)
    if (!at_bytes(p, 16)) return false;
  return true;
}

}  // namespace

size_t layer_norm_bwd_workspace_bytes(int64_t rows, int D) {
  return rows <= 0 || D <= 0 ? 0 : sizeof(float) * kParts * 2 * static_cast<size_t>(D);
}

cudaError_t layer_norm_fwd_launch(const NormArgs& a, cudaStream_t st) {
  const bool vec = vectors(a.D, a.dtype, {a.x, a.residual, a.sum, a.y, a.weight, a.bias});
  if (a.dtype == SANATAN_F32) return vec ? fwd<float, true>(a, st) : fwd<float, false>(a, st);
  return vec ? fwd<__nv_bfloat16, true>(a, st) : fwd<__nv_bfloat16, false>(a, st);
}

cudaError_t layer_norm_bwd_launch(const NormBwdArgs& a, cudaStream_t st) {
  if (a.rows == 0) {
    const size_t row = static_cast<size_t>(a.D) * sizeof(float);
    cudaError_t e = a.dweight != nullptr ? cudaMemsetAsync(a.dweight, 0, row, st) : cudaSuccess;
    if (e == cudaSuccess && a.dbias != nullptr) e = cudaMemsetAsync(a.dbias, 0, row, st);
    return e;
  }
  const bool vec = vectors(a.D, a.dtype, {a.s, a.dy, a.ds, a.dx, a.weight});
  if (a.dtype == SANATAN_F32) return vec ? bwd<float, true>(a, st) : bwd<float, false>(a, st);
  return vec ? bwd<__nv_bfloat16, true>(a, st) : bwd<__nv_bfloat16, false>(a, st);
}

}  // namespace sanatan
