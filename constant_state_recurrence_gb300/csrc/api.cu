// C ABI of libsanatan.so: host-side validation and dispatch (see sanatan.h).
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "sanatan_internal.h"

namespace {

using namespace sanatan;

constexpr int kAbiVersion = 2;
constexpr int kMaxPower = 8;   // largest p of sanatan_power_fwd

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
bool ok_nullable(const void* p) { return p == nullptr || aligned16(p); }
// Where an element of `size` bytes may start: for what kernels touch element by element.
bool at_element(const void* p, size_t size) {
  return reinterpret_cast<uintptr_t>(p) % size == 0;
}
bool ok_floats(const float* p) { return p != nullptr && at_element(p, 4); }
bool ok_dtype(int t) { return t == SANATAN_F32 || t == SANATAN_BF16; }

int from_cuda(cudaError_t e) { return e == cudaSuccess ? SANATAN_OK : SANATAN_ERR_CUDA; }

// The kernels are built for sm_103a only; refuse any other device before a
// launch could fail with "no kernel image".
int check_arch() {
  static int cached[64];  // 0 unknown, 1 ok, 2 wrong arch
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SANATAN_ERR_CUDA;
  if (dev >= 0 && dev < 64 && cached[dev] != 0) return cached[dev] == 1 ? SANATAN_OK : SANATAN_ERR_ARCH;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return SANATAN_ERR_CUDA;
  const bool ok = (major == 10 && minor == 3);
  if (dev >= 0 && dev < 64) cached[dev] = ok ? 1 : 2;
  return ok ? SANATAN_OK : SANATAN_ERR_ARCH;
}

int check_sizes(int B, int H, int T, int d, int dv) {
  if (B < 0 || H < 0 || T < 0 || d < 0 || dv < 0) return SANATAN_ERR_INVALID;
  if (d != 64 || dv != 64) return SANATAN_ERR_UNSUPPORTED;
  // Element counts index with 64-bit arithmetic; CTA counts must fit a grid.
  if (static_cast<int64_t>(B) * H > (1LL << 31) - 1) return SANATAN_ERR_UNSUPPORTED;
  return SANATAN_OK;
}

int check_params(const float* gamma, const float* omega, const float* phi) {
  if (!ok_ptr(gamma) || !ok_ptr(omega) || !ok_ptr(phi)) return SANATAN_ERR_INVALID;
  return SANATAN_OK;
}

int check_scan(int dtype, int gate, int B, int T, int D) {
  if (!ok_dtype(dtype)) return SANATAN_ERR_INVALID;
  if (gate != SANATAN_GATE_LOG && gate != SANATAN_GATE_SIGMOID) return SANATAN_ERR_INVALID;
  if (B < 0 || T < 0 || D < 0) return SANATAN_ERR_INVALID;
  // Elements index with 64-bit arithmetic; thread blocks must fit a grid.
  if (static_cast<int64_t>(B) * D > (1LL << 31) - 1) return SANATAN_ERR_UNSUPPORTED;
  // Token and channel indexes are ints, also those of a tile that reaches past the end.
  if (T > (1 << 30) || D > (1 << 30)) return SANATAN_ERR_UNSUPPORTED;
  return SANATAN_OK;
}

struct Range {
  const void* p;
  size_t n;
};

// Whether two ranges share bytes (null: no range).
bool overlap(const void* a, size_t n, const void* b, size_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && n > 0 && m > 0 && x < y + m && y < x + n;
}

// Whether an output shares bytes with an input or another output.  may[k] = {output, input}
// are pairs that may be one and the same tensor.
struct Pair {
  int out, in;
};
bool clash(std::initializer_list<Range> out, std::initializer_list<Range> in,
           std::initializer_list<Pair> may = {}) {
  int o = 0;
  for (const Range* x = out.begin(); x != out.end(); ++x, ++o) {
    int i = 0;
    for (const Range* y = in.begin(); y != in.end(); ++y, ++i) {
      bool same = false;
      for (const Pair& m : may) same |= m.out == o && m.in == i && x->p == y->p;
      if (!same && overlap(x->p, x->n, y->p, y->n)) return true;
    }
    for (const Range* y = out.begin(); y != x; ++y)
      if (overlap(x->p, x->n, y->p, y->n)) return true;
  }
  return false;
}

size_t size_of(int dtype) { return dtype == SANATAN_F32 ? 4 : 2; }

// Pointers that may start at any element: null only where `nullable`.
bool at_elements(std::initializer_list<const void*> all, size_t size, bool nullable = false) {
  for (const void* p : all)
    if ((p == nullptr && !nullable) || !at_element(p, size)) return false;
  return true;
}

// Bytes of `rows` rows of `width` values, ld between two.
size_t span(int64_t rows, int64_t ld, int64_t width, size_t size) {
  return rows <= 0 ? 0 : (static_cast<size_t>(rows - 1) * ld + width) * size;
}

// Sizes of the layers over [B, T, D] (width: values of the widest row; N: states).
int check_layer(int dtype, int B, int T, int D, int64_t widest, int N) {
  if (!ok_dtype(dtype) || B < 0 || T < 0 || D < 0) return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * D > (1LL << 31) - 1) return SANATAN_ERR_UNSUPPORTED;
  if (T > (1 << 30) || D > (1 << 30)) return SANATAN_ERR_UNSUPPORTED;
  const double tokens = static_cast<double>(B) * (T + 16.0);
  // Offsets fit 60 bits; a thread block holds at least 128 of a launch's items.
  if (tokens * widest > 1e18 || tokens * D * N > 1e18) return SANATAN_ERR_UNSUPPORTED;
  if (tokens / 16 * D / 128 > 2e9 || tokens * N / 128 > 2e9) return SANATAN_ERR_UNSUPPORTED;
  return SANATAN_OK;
}

int check_norm(int dtype, int64_t rows, int D) {
  if (!ok_dtype(dtype) || rows < 0 || D < 0) return SANATAN_ERR_INVALID;
  return rows > (1LL << 31) - 1 || D > (1 << 30) ? SANATAN_ERR_UNSUPPORTED : SANATAN_OK;
}

int check_conv(int dtype, int act, int B, int T, int D, int K, int64_t ldx) {
  if (act != SANATAN_ACT_NONE && act != SANATAN_ACT_SILU) return SANATAN_ERR_INVALID;
  if (K < 1 || ldx < D) return SANATAN_ERR_INVALID;
  if (int s = check_layer(dtype, B, T, D, ldx, 1)) return s;
  return K > kConvTaps ? SANATAN_ERR_UNSUPPORTED : SANATAN_OK;
}

// The selective scan's inputs, shared by its calls (T = 1: the step, lens and h0 null).
int check_selective(const SelectiveArgs& a) {
  if (a.N < 1 || a.ldb < a.N || a.ldc < a.N || (a.z != nullptr && a.ldz < a.D))
    return SANATAN_ERR_INVALID;
  const int64_t widest = std::max(std::max(a.ldb, a.ldc), a.z != nullptr ? a.ldz : 0);
  if (int s = check_layer(a.dtype, a.B, a.T, a.D, std::max<int64_t>(widest, a.D),
                          std::min(a.N, kSelectiveStates)))
    return s;
  if (a.N > kSelectiveStates) return SANATAN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(a.B) * a.D == 0) return SANATAN_OK;
  const size_t e = size_of(a.dtype);
  if (!at_elements({a.A}, 4) || !at_elements({a.skip, a.dt_bias, a.h0, a.h_out, a.marks}, 4, true) ||
      !at_elements({a.lens}, 8, true) || !at_elements({a.z}, e, true))
    return SANATAN_ERR_INVALID;
  if (a.T > 0 && !at_elements({a.u, a.dt, a.Bm, a.Cm}, e)) return SANATAN_ERR_INVALID;
  return SANATAN_OK;
}

// Argument checks and launch of the state cache's two directions.
int state_cache(float* state, float* exact, int layers, int B, int64_t inner, int64_t exact_inner,
                const int64_t* pages, int64_t num_pages, int fmt, void* codes, float* scales,
                float* exact_cache, bool write, void* stream) {
  if (fmt != SANATAN_CACHE_INT8 && fmt != SANATAN_CACHE_E4M3) return SANATAN_ERR_INVALID;
  if (layers < 0 || B < 0 || inner < 0 || exact_inner < 0 || num_pages < 0)
    return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(layers) * B == 0 || (inner == 0 && exact_inner == 0) || num_pages == 0)
    return SANATAN_OK;
  if (pages == nullptr || !at_element(pages, 8)) return SANATAN_ERR_INVALID;
  if (inner > 0 && (!ok_floats(state) || !ok_ptr(codes) || !ok_ptr(scales)))
    return SANATAN_ERR_INVALID;
  if (exact_inner > 0 && (!ok_floats(exact) || !ok_ptr(exact_cache))) return SANATAN_ERR_INVALID;
  // Thread blocks must fit a grid, and the largest offset 63 bits.
  const int64_t most = (1LL << 31) - 1;
  if (inner > (1LL << 40) || exact_inner > (1LL << 40) || num_pages > most)
    return SANATAN_ERR_UNSUPPORTED;
  const int64_t blocks = state_cache_blocks(inner);
  if (blocks > most / (static_cast<int64_t>(layers) * B)) return SANATAN_ERR_UNSUPPORTED;
  if (static_cast<double>(num_pages) * layers * (inner + exact_inner + 64.0) > 1e18 ||
      static_cast<double>(B) * layers * (inner + exact_inner + 64.0) > 1e18)
    return SANATAN_ERR_UNSUPPORTED;
  if (int s = check_arch()) return s;
  CacheArgs a;
  a.state = state;
  a.exact = exact;
  a.layers = layers;
  a.B = B;
  a.inner = inner;
  a.exact_inner = exact_inner;
  a.pages = pages;
  a.num_pages = num_pages;
  a.fmt = fmt;
  a.codes = codes;
  a.scales = scales;
  a.exact_cache = exact_cache;
  a.blocks = static_cast<unsigned>(blocks);
  return from_cuda(state_cache_launch(a, write, static_cast<cudaStream_t>(stream)));
}

}  // namespace

namespace sanatan {
ProfileEvents& profile_events() {
  static thread_local ProfileEvents ev;
  return ev;
}
}  // namespace sanatan

extern "C" {

const char* sanatan_status_string(int status) {
  switch (status) {
    case SANATAN_OK: return "ok";
    case SANATAN_ERR_INVALID: return "invalid argument (null or misaligned pointer, negative size, bad enum)";
    case SANATAN_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case SANATAN_ERR_CUDA: return "CUDA runtime error";
    case SANATAN_ERR_ARCH: return "device is not sm_103 (GB300)";
    case SANATAN_ERR_TIMEOUT: return "device-side bounded wait timed out";
    default: return "unknown status";
  }
}

int sanatan_abi_version(void) { return kAbiVersion; }

size_t sanatan_state_bytes(int layers, int heads, int d, int dv) {
  if (layers < 0 || heads < 0 || d < 0 || dv < 0) return 0;
  return static_cast<size_t>(layers) * heads * (6ull * d * dv + 6ull * d) * sizeof(float);
}

int sanatan_featurize(const void* u, int u_dtype, const float* gamma, const float* omega,
                      const float* phi, int B, int H, int T, int d, int64_t pos0, void* out,
                      int out_dtype, void* stream) {
  if (!ok_dtype(u_dtype) || !ok_dtype(out_dtype)) return SANATAN_ERR_INVALID;
  if (B < 0 || H < 0 || T < 0 || d <= 0) return SANATAN_ERR_INVALID;
  if (d != 64) return SANATAN_ERR_UNSUPPORTED;
  const int64_t n = static_cast<int64_t>(B) * H * T;
  if (n == 0) return SANATAN_OK;
  if (!ok_ptr(u) || !ok_ptr(out)) return SANATAN_ERR_INVALID;
  if (int s = check_params(gamma, omega, phi)) return s;
  if (n * d / 256 + 1 > 0x7fffffffLL) return SANATAN_ERR_UNSUPPORTED;
  if (int s = check_arch()) return s;
  return from_cuda(featurize_launch(u, u_dtype, gamma, omega, phi, B, H, T, d, pos0, out,
                                    out_dtype, static_cast<cudaStream_t>(stream)));
}

int sanatan_rate_from_raw(const float* lambda_raw, int n, float scale, float* phi, void* stream) {
  if (n < 0) return SANATAN_ERR_INVALID;
  if (n == 0) return SANATAN_OK;
  if (!ok_ptr(lambda_raw) || !ok_ptr(phi)) return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  return from_cuda(rate_launch(lambda_raw, nullptr, n, scale, phi,
                               static_cast<cudaStream_t>(stream)));
}

int sanatan_rate_from_raw_bwd(const float* lambda_raw, const float* dphi, int n, float scale,
                              float* dlambda_raw, void* stream) {
  if (n < 0) return SANATAN_ERR_INVALID;
  if (n == 0) return SANATAN_OK;
  if (!ok_ptr(lambda_raw) || !ok_ptr(dphi) || !ok_ptr(dlambda_raw)) return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  return from_cuda(rate_launch(lambda_raw, dphi, n, scale, dlambda_raw,
                               static_cast<cudaStream_t>(stream)));
}

float sanatan_eps_raw(float eps, int d, int convention) {
  if (d <= 0) return -1.0f;
  if (convention == 0) return (4.0f * static_cast<float>(d) + 1e-6f) * eps;
  if (convention == 1) return (4.0f * static_cast<float>(d) * 1e-6f) * eps;
  return -1.0f;
}

size_t sanatan_chunk_fwd_workspace_size(int B, int H, int T, int d, int dv, int in_dtype) {
  if (B < 0 || H < 0 || T < 0 || d != 64 || dv != 64) return 0;
  if (in_dtype != SANATAN_BF16) return 0;
  return chunk_fwd_tc_workspace_bytes(B, H, T);
}

int sanatan_chunk_fwd_plan(int B, int H, int T, int in_dtype, int has_initial_state,
                           int* segments, int* launches) {
  if (!ok_dtype(in_dtype) || B < 0 || H < 0 || T < 0 || segments == nullptr || launches == nullptr)
    return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * H == 0) {
    *segments = 0;
    *launches = 0;
    return SANATAN_OK;
  }
  if (in_dtype == SANATAN_F32) {
    *segments = 1;
    *launches = 1;
    return SANATAN_OK;
  }
  const int nseg = tc_segments(B, H, T);
  *segments = nseg;
  (void)has_initial_state;
  *launches = 1 + (nseg > 1 ? 1 : 0);
  return SANATAN_OK;
}

int sanatan_chunk_fwd(const void* q, const void* k, const void* v, int in_dtype,
                      const float* gamma, const float* omega, const float* phi, int B, int H,
                      int T, int d, int dv, int64_t pos0, float eps, const float* S0,
                      const float* z0, float* o, float* D, float* S_out, float* z_out,
                      void* workspace, size_t workspace_bytes, void* stream) {
  return sanatan::chunk_fwd_checked(q, k, v, in_dtype, gamma, omega, phi, B, H, T, d, dv, pos0,
                                    eps, S0, z0, o, D, S_out, z_out, workspace, workspace_bytes,
                                    stream, false);
}

}  // extern "C"

namespace sanatan {
// Argument checks and dispatch of sanatan_chunk_fwd.  With `fewer_segments`
// a workspace smaller than sanatan_chunk_fwd_workspace_size is accepted and
// the tensor-core path splits sequences into as many segments as it holds.
int chunk_fwd_checked(const void* q, const void* k, const void* v, int in_dtype,
                      const float* gamma, const float* omega, const float* phi, int B, int H,
                      int T, int d, int dv, int64_t pos0, float eps, const float* S0,
                      const float* z0, float* o, float* D, float* S_out, float* z_out,
                      void* workspace, size_t workspace_bytes, void* stream, bool fewer_segments) {
  if (!ok_dtype(in_dtype)) return SANATAN_ERR_INVALID;
  if (int s = check_sizes(B, H, T, d, dv)) return s;
  if ((S0 == nullptr) != (z0 == nullptr)) return SANATAN_ERR_INVALID;
  if ((S_out == nullptr) != (z_out == nullptr)) return SANATAN_ERR_INVALID;
  if (!ok_nullable(S0) || !ok_nullable(z0) || !ok_nullable(S_out) || !ok_nullable(z_out) ||
      !ok_nullable(D) || !ok_nullable(workspace))
    return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * H == 0) return SANATAN_OK;
  if (T > 0 && (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o))) return SANATAN_ERR_INVALID;
  if (int s = check_params(gamma, omega, phi)) return s;
  if (!fewer_segments &&
      workspace_bytes < sanatan_chunk_fwd_workspace_size(B, H, T, d, dv, in_dtype))
    return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  ChunkFwdArgs a{q, k, v, in_dtype, gamma, omega, phi, B, H, T, d, dv, pos0, eps,
                 S0, z0, o, D, S_out, z_out, workspace, workspace_bytes};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (in_dtype == SANATAN_BF16) return from_cuda(chunk_fwd_tc_launch(a, st));
  return from_cuda(chunk_fwd_simt_launch(a, st));
}
}  // namespace sanatan

extern "C" {

size_t sanatan_chunk_bwd_workspace_size(int B, int H, int T, int d, int dv, int in_dtype) {
  if (B < 0 || H < 0 || T < 0 || d != 64 || dv != 64) return 0;
  if (in_dtype != SANATAN_BF16) return 0;
  return chunk_bwd_tc_workspace_bytes(B, H, T);
}

int sanatan_chunk_bwd(const void* q, const void* k, const void* v, int in_dtype,
                      const float* gamma, const float* omega, const float* phi, int B, int H,
                      int T, int d, int dv, int64_t pos0, float eps, const float* S0,
                      const float* z0, const float* o, const float* D, const void* dO,
                      int grad_dtype, void* dq, void* dk, void* dv_out, float* dgamma,
                      float* domega, float* dphi, void* workspace, size_t workspace_bytes,
                      const void* fwd_workspace, size_t fwd_workspace_bytes, void* stream) {
  if (!ok_dtype(in_dtype) || !ok_dtype(grad_dtype)) return SANATAN_ERR_INVALID;
  if (!ok_nullable(fwd_workspace)) return SANATAN_ERR_INVALID;
  if (int s = check_sizes(B, H, T, d, dv)) return s;
  if ((S0 == nullptr) != (z0 == nullptr)) return SANATAN_ERR_INVALID;
  if (!ok_nullable(S0) || !ok_nullable(z0) || !ok_nullable(dphi) || !ok_nullable(workspace))
    return SANATAN_ERR_INVALID;
  if (H > 0 && (!ok_ptr(dgamma) || !ok_ptr(domega))) return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * H * T > 0 &&
      (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) || !ok_ptr(D) || !ok_ptr(dO) ||
       !ok_ptr(dq) || !ok_ptr(dk) || !ok_ptr(dv_out)))
    return SANATAN_ERR_INVALID;
  if (H > 0) {
    if (int s = check_params(gamma, omega, phi)) return s;
  }
  if (workspace_bytes < sanatan_chunk_bwd_workspace_size(B, H, T, d, dv, in_dtype))
    return SANATAN_ERR_INVALID;
  if (H == 0) return SANATAN_OK;
  if (int s = check_arch()) return s;
  ChunkBwdArgs a{};
  a.f = ChunkFwdArgs{q, k, v, in_dtype, gamma, omega, phi, B, H, T, d, dv, pos0, eps,
                     S0, z0, nullptr, nullptr, nullptr, nullptr, workspace, workspace_bytes};
  a.o = o;
  a.Dn = D;
  a.dO = dO;
  a.grad_dtype = grad_dtype;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv_out;
  a.dgamma = dgamma;
  a.domega = domega;
  a.dphi = dphi;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.fwd_workspace = fwd_workspace;
  a.fwd_workspace_bytes = fwd_workspace == nullptr ? 0 : fwd_workspace_bytes;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (in_dtype == SANATAN_BF16) return from_cuda(chunk_bwd_tc_launch(a, st));
  return from_cuda(chunk_bwd_simt_launch(a, st));
}

size_t sanatan_power_fwd_workspace_size(int B, int H, int T, int d, int dv) {
  if (B < 0 || H < 0 || T < 0 || d != 64 || dv != 64) return 0;
  return pow_fwd_tc_workspace_bytes(B, H, T);
}

int sanatan_power_fwd(const void* q, const void* k, const void* v, const float* gamma,
                      const float* omega, const float* phi, int B, int H, int T, int d, int dv,
                      int64_t pos0, int p, float eps, float* o, float* D, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (int s = check_sizes(B, H, T, d, dv)) return s;
  if (p < 1) return SANATAN_ERR_INVALID;
  if (p > kMaxPower) return SANATAN_ERR_UNSUPPORTED;
  if (!ok_nullable(D)) return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * H == 0 || T == 0) return SANATAN_OK;
  if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) || !ok_ptr(workspace))
    return SANATAN_ERR_INVALID;
  if (int s = check_params(gamma, omega, phi)) return s;
  if (workspace_bytes < pow_fwd_tc_workspace_bytes(B, H, T)) return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * H * ((T + 127) / 128) > 0x3fffffffLL) return SANATAN_ERR_UNSUPPORTED;
  if (int s = check_arch()) return s;
  PowFwdArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.gamma = gamma;
  a.omega = omega;
  a.phi = phi;
  a.B = B;
  a.H = H;
  a.T = T;
  a.pos0 = pos0;
  a.p = p;
  a.eps = eps;
  a.o = o;
  a.D = D;
  a.workspace = workspace;
  return from_cuda(pow_fwd_tc_launch(a, static_cast<cudaStream_t>(stream)));
}

int sanatan_ablation_fwd(const void* q, const void* k, const void* v, const float* gamma,
                         const float* omega, const float* phi, int B, int H, int T, int d,
                         int dv, int64_t pos0, int p, int channels, float shift, float eps,
                         float* o, float* D, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (int s = check_sizes(B, H, T, d, dv)) return s;
  if (channels != 3 && channels != 4) return SANATAN_ERR_INVALID;
  if (!(shift >= 0.0f) || (channels == 4 && shift != 0.0f)) return SANATAN_ERR_INVALID;
  if (p < 1) return SANATAN_ERR_INVALID;
  if (p != 1 && p != 2 && p != 4) return SANATAN_ERR_UNSUPPORTED;
  if (!ok_nullable(D)) return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * H == 0 || T == 0) return SANATAN_OK;
  if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) || !ok_ptr(workspace))
    return SANATAN_ERR_INVALID;
  if (int s = check_params(gamma, omega, phi)) return s;
  if (workspace_bytes < pow_fwd_tc_workspace_bytes(B, H, T)) return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * H * ((T + 127) / 128) > 0x3fffffffLL) return SANATAN_ERR_UNSUPPORTED;
  if (int s = check_arch()) return s;
  PowFwdArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.gamma = gamma;
  a.omega = omega;
  a.phi = phi;
  a.B = B;
  a.H = H;
  a.T = T;
  a.pos0 = pos0;
  a.p = p;
  a.eps = eps;
  a.o = o;
  a.D = D;
  a.workspace = workspace;
  return from_cuda(ablation_fwd_tc_launch(a, channels, shift, static_cast<cudaStream_t>(stream)));
}

size_t sanatan_power_bwd_workspace_size(int B, int H, int T, int d, int dv) {
  if (B < 0 || H < 0 || T < 0 || d != 64 || dv != 64) return 0;
  return pow_bwd_tc_workspace_bytes(B, H, T);
}

int sanatan_power_bwd(const void* q, const void* k, const void* v, const float* gamma,
                      const float* omega, const float* phi, int B, int H, int T, int d, int dv,
                      int64_t pos0, int p, float eps, const float* o, const float* D,
                      const void* dO, int grad_dtype, void* dq, void* dk, void* dv_out,
                      float* dgamma, float* domega, float* dphi, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (int s = check_sizes(B, H, T, d, dv)) return s;
  if (p < 1 || !ok_dtype(grad_dtype)) return SANATAN_ERR_INVALID;
  if (p > kMaxPower) return SANATAN_ERR_UNSUPPORTED;
  if (H > 0 && (!ok_ptr(dgamma) || !ok_ptr(domega) || !ok_nullable(dphi)))
    return SANATAN_ERR_INVALID;
  if (H > 0) {
    if (int s = check_params(gamma, omega, phi)) return s;
  }
  if (static_cast<int64_t>(B) * H > 0 && T > 0) {
    if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) || !ok_ptr(D) || !ok_ptr(dO) ||
        !ok_ptr(dq) || !ok_ptr(dk) || !ok_ptr(dv_out) || !ok_ptr(workspace))
      return SANATAN_ERR_INVALID;
    if (workspace_bytes < pow_bwd_tc_workspace_bytes(B, H, T)) return SANATAN_ERR_INVALID;
    if (static_cast<int64_t>(B) * H * ((T + 127) / 128) > 0x3fffffffLL)
      return SANATAN_ERR_UNSUPPORTED;
  }
  if (H == 0) return SANATAN_OK;
  if (int s = check_arch()) return s;
  PowBwdArgs a;
  a.f.q = q;
  a.f.k = k;
  a.f.v = v;
  a.f.gamma = gamma;
  a.f.omega = omega;
  a.f.phi = phi;
  a.f.B = B;
  a.f.H = H;
  a.f.T = T;
  a.f.pos0 = pos0;
  a.f.p = p;
  a.f.eps = eps;
  a.f.workspace = workspace;
  a.o = o;
  a.D = D;
  a.dO = dO;
  a.grad_dtype = grad_dtype;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv_out;
  a.dgamma = dgamma;
  a.domega = domega;
  a.dphi = dphi;
  return from_cuda(pow_bwd_tc_launch(a, static_cast<cudaStream_t>(stream)));
}

int sanatan_set_profile_events(void* start, void* stop) {
  if ((start == nullptr) != (stop == nullptr)) return SANATAN_ERR_INVALID;
  profile_events().start = static_cast<cudaEvent_t>(start);
  profile_events().stop = static_cast<cudaEvent_t>(stop);
  return SANATAN_OK;
}

int sanatan_device_status(void* stream) {
  if (int s = check_arch()) return s;
  const int h = tc_read_and_clear_error(static_cast<cudaStream_t>(stream));
  const int hb = bwd_tc_read_and_clear_error(static_cast<cudaStream_t>(stream));
  const int hp = pow_tc_read_and_clear_error(static_cast<cudaStream_t>(stream));
  const int hpb = pow_bwd_tc_read_and_clear_error(static_cast<cudaStream_t>(stream));
  const int hs = stack_read_and_clear_error(static_cast<cudaStream_t>(stream));
  const int hg = scan_fwd_read_and_clear_error(static_cast<cudaStream_t>(stream));
  const int hgb = scan_bwd_read_and_clear_error(static_cast<cudaStream_t>(stream));
  if (h < 0 || hb < 0 || hp < 0 || hpb < 0 || hs < 0 || hg < 0 || hgb < 0) return SANATAN_ERR_CUDA;
  if (hb || hp || hpb || hs || hg || hgb) return SANATAN_ERR_TIMEOUT;
  return h ? SANATAN_ERR_TIMEOUT : SANATAN_OK;
}

size_t sanatan_state_bytes_harmonic(int layers, int heads, int d, int dv, int harmonics) {
  if (layers < 0 || heads < 0 || d < 0 || dv < 0 || harmonics < 1) return 0;
  const size_t F = static_cast<size_t>(2 * (2 * harmonics + 1)) * d;
  return static_cast<size_t>(layers) * heads * (F * dv + F) * sizeof(float);
}

int sanatan_featurize_harmonic(const void* u, int u_dtype, const float* gamma, const float* omega,
                               const float* phi, int B, int H, int T, int d, int64_t pos0,
                               int harmonics, void* out, int out_dtype, void* stream) {
  if (!ok_dtype(u_dtype) || !ok_dtype(out_dtype)) return SANATAN_ERR_INVALID;
  if (B < 0 || H < 0 || T < 0 || d <= 0 || harmonics < 1) return SANATAN_ERR_INVALID;
  if (d != 64 || harmonics > 3) return SANATAN_ERR_UNSUPPORTED;
  const int64_t n = static_cast<int64_t>(B) * H * T;
  if (n == 0) return SANATAN_OK;
  if (!ok_ptr(u) || !ok_ptr(out)) return SANATAN_ERR_INVALID;
  if (int s = check_params(gamma, omega, phi)) return s;
  if (n * d / 256 + 1 > 0x7fffffffLL) return SANATAN_ERR_UNSUPPORTED;
  if (int s = check_arch()) return s;
  HarmonicFeatArgs a{u, u_dtype, gamma, omega, phi, B, H, T, pos0, harmonics, out, out_dtype};
  return from_cuda(featurize_harmonic_launch(a, static_cast<cudaStream_t>(stream)));
}

int sanatan_chunk_fwd_harmonic(const void* q, const void* k, const void* v, int in_dtype,
                               const float* gamma, const float* omega, const float* phi, int B,
                               int H, int T, int d, int dv, int64_t pos0, int harmonics,
                               float eps, const float* S0, const float* z0, float* o, float* D,
                               float* S_out, float* z_out, void* stream) {
  if (!ok_dtype(in_dtype) || harmonics < 1) return SANATAN_ERR_INVALID;
  if (int s = check_sizes(B, H, T, d, dv)) return s;
  if (harmonics > 3) return SANATAN_ERR_UNSUPPORTED;
  if ((S0 == nullptr) != (z0 == nullptr)) return SANATAN_ERR_INVALID;
  if ((S_out == nullptr) != (z_out == nullptr)) return SANATAN_ERR_INVALID;
  if (!ok_nullable(S0) || !ok_nullable(z0) || !ok_nullable(S_out) || !ok_nullable(z_out) ||
      !ok_nullable(D))
    return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * H == 0) return SANATAN_OK;
  if (T > 0 && (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o))) return SANATAN_ERR_INVALID;
  if (int s = check_params(gamma, omega, phi)) return s;
  if (int s = check_arch()) return s;
  ChunkFwdArgs a{q, k, v, in_dtype, gamma, omega, phi, B, H, T, d, dv, pos0, eps,
                 S0, z0, o, D, S_out, z_out, nullptr, 0};
  return from_cuda(chunk_fwd_harmonic_launch(a, harmonics, static_cast<cudaStream_t>(stream)));
}

size_t sanatan_chunk_bwd_harmonic_workspace_size(int B, int H, int T, int d, int dv,
                                                 int harmonics) {
  if (B < 0 || H < 0 || T < 0 || d != 64 || dv != 64 || harmonics < 1 || harmonics > 3) return 0;
  return chunk_bwd_harmonic_workspace_bytes(B, H, T, harmonics);
}

int sanatan_chunk_bwd_harmonic(const void* q, const void* k, const void* v, int in_dtype,
                               const float* gamma, const float* omega, const float* phi, int B,
                               int H, int T, int d, int dv, int64_t pos0, int harmonics,
                               float eps, const float* S0, const float* z0, const float* o,
                               const float* D, const void* dO, int grad_dtype, void* dq, void* dk,
                               void* dv_out, float* dgamma, float* domega, float* dphi,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!ok_dtype(in_dtype) || !ok_dtype(grad_dtype) || harmonics < 1) return SANATAN_ERR_INVALID;
  if (int s = check_sizes(B, H, T, d, dv)) return s;
  if (harmonics > 3) return SANATAN_ERR_UNSUPPORTED;
  if ((S0 == nullptr) != (z0 == nullptr)) return SANATAN_ERR_INVALID;
  if (!ok_nullable(S0) || !ok_nullable(z0) || !ok_nullable(dphi) || !ok_nullable(workspace))
    return SANATAN_ERR_INVALID;
  if (H > 0 && (!ok_ptr(dgamma) || !ok_ptr(domega))) return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * H * T > 0 &&
      (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) || !ok_ptr(D) || !ok_ptr(dO) ||
       !ok_ptr(dq) || !ok_ptr(dk) || !ok_ptr(dv_out)))
    return SANATAN_ERR_INVALID;
  if (H > 0) {
    if (int s = check_params(gamma, omega, phi)) return s;
  }
  const size_t need = sanatan_chunk_bwd_harmonic_workspace_size(B, H, T, d, dv, harmonics);
  if (workspace_bytes < need || (need > 0 && workspace == nullptr)) return SANATAN_ERR_INVALID;
  if (H == 0) return SANATAN_OK;
  if (int s = check_arch()) return s;
  ChunkBwdArgs a{};
  a.f = ChunkFwdArgs{q, k, v, in_dtype, gamma, omega, phi, B, H, T, d, dv, pos0, eps,
                     S0, z0, nullptr, nullptr, nullptr, nullptr, nullptr, 0};
  a.o = o;
  a.Dn = D;
  a.dO = dO;
  a.grad_dtype = grad_dtype;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv_out;
  a.dgamma = dgamma;
  a.domega = domega;
  a.dphi = dphi;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  return from_cuda(
      chunk_bwd_harmonic_launch(a, harmonics, static_cast<cudaStream_t>(stream)));
}

int sanatan_decode_step_harmonic(float* S, float* z, const float* q, const float* k,
                                 const float* v, const float* gamma, const float* omega,
                                 const float* phi, const int64_t* pos, int N, int G, int d, int dv,
                                 int harmonics, float eps, float* o, void* stream) {
  if (N < 0 || G <= 0 || d < 0 || dv < 0 || harmonics < 1) return SANATAN_ERR_INVALID;
  if (d != 64 || dv != 64 || harmonics > 3) return SANATAN_ERR_UNSUPPORTED;
  if (N == 0) return SANATAN_OK;
  if (!ok_ptr(S) || !ok_ptr(z) || !ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(pos) ||
      !ok_ptr(o))
    return SANATAN_ERR_INVALID;
  if (int s = check_params(gamma, omega, phi)) return s;
  if (static_cast<int64_t>(N) * 4 > 0x7fffffffLL) return SANATAN_ERR_UNSUPPORTED;
  if (int s = check_arch()) return s;
  return from_cuda(decode_harmonic_launch(S, z, q, k, v, gamma, omega, phi, pos, N, G, eps,
                                          harmonics, o, static_cast<cudaStream_t>(stream)));
}

size_t sanatan_stack_decode_workspace_size(int B, int heads, int d) {
  if (B < 0 || heads < 0 || d != 64) return 0;
  return stack_workspace_bytes(B, heads, d);
}

int sanatan_stack_decode_step(float* x, const float* Wqkv, const float* Wo, float* S, float* z,
                              const float* gamma, const float* omega, const float* phi,
                              const int64_t* pos, int B, int L, int heads, int d, float eps,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || L < 0 || heads < 0 || d < 0) return SANATAN_ERR_INVALID;
  if (d != 64 || B > stack_max_batch() || (heads * d) % 128 != 0) return SANATAN_ERR_UNSUPPORTED;
  if (B == 0 || L == 0 || heads == 0) return SANATAN_OK;
  if (!ok_ptr(x) || !ok_ptr(Wqkv) || !ok_ptr(Wo) || !ok_ptr(S) || !ok_ptr(z) || !ok_ptr(pos) ||
      !ok_ptr(workspace))
    return SANATAN_ERR_INVALID;
  if (int s = check_params(gamma, omega, phi)) return s;
  if (workspace_bytes < stack_workspace_bytes(B, heads, d)) return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  StackArgs a{x, Wqkv, Wo, S, z, gamma, omega, phi, pos, B, L, heads, eps, workspace};
  return from_cuda(stack_decode_launch(a, static_cast<cudaStream_t>(stream)));
}

int sanatan_selftest_wait_timeout(uint64_t timeout_ns, int arrive, void* stream) {
  if (timeout_ns < 1000ull || timeout_ns > 1000000000ull) return SANATAN_ERR_INVALID;
  if (arrive != 0 && arrive != 1) return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  return from_cuda(tc_timeout_probe_launch(timeout_ns, arrive, static_cast<cudaStream_t>(stream)));
}

int sanatan_decode_step(float* S, float* z, const float* q, const float* k, const float* v,
                        const float* gamma, const float* omega, const float* phi,
                        const int64_t* pos, int N, int G, int d, int dv, float eps, float* o,
                        void* stream) {
  if (N < 0 || G <= 0 || d < 0 || dv < 0) return SANATAN_ERR_INVALID;
  if (d != 64 || dv != 64) return SANATAN_ERR_UNSUPPORTED;
  if (N == 0) return SANATAN_OK;
  if (!ok_ptr(S) || !ok_ptr(z) || !ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(pos) ||
      !ok_ptr(o))
    return SANATAN_ERR_INVALID;
  if (int s = check_params(gamma, omega, phi)) return s;
  if (int s = check_arch()) return s;
  return from_cuda(decode_step_launch(S, z, q, k, v, gamma, omega, phi, pos, N, G, eps, o,
                                      static_cast<cudaStream_t>(stream)));
}

size_t sanatan_gated_scan_marks_size(int B, int T, int D) {
  if (B < 0 || T < 0 || D < 0) return 0;
  return static_cast<size_t>(B) * ((static_cast<size_t>(T) + kScanMark - 1) / kScanMark) * D *
         sizeof(float);
}

int sanatan_gated_scan_fwd(const void* x, const void* g, int dtype, int gate, const int64_t* lens,
                           int B, int T, int D, const float* h0, void* y, float* h_out,
                           float* marks, void* stream) {
  if (int s = check_scan(dtype, gate, B, T, D)) return s;
  if (!ok_nullable(lens) || !ok_nullable(h0) || !ok_nullable(h_out) || !ok_nullable(marks))
    return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * D == 0) return SANATAN_OK;
  if (T > 0 && (!ok_ptr(x) || !ok_ptr(g) || !ok_ptr(y))) return SANATAN_ERR_INVALID;
  if (T == 0 && h_out == nullptr) return SANATAN_OK;
  const size_t state = static_cast<size_t>(B) * D * 4;
  const size_t all = static_cast<size_t>(B) * T * D * (dtype == SANATAN_F32 ? 4 : 2);
  const size_t nm = sanatan_gated_scan_marks_size(B, T, D);
  const size_t len = static_cast<size_t>(B) * 8;
  const Range in[] = {{x, all}, {g, all}, {lens, len}, {h0, state}};
  const Range out[] = {{y, all}, {marks, nm}, {h_out, state}};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 4; ++i)  // (h_out may be h0)
      if (overlap(out[o].p, out[o].n, in[i].p, in[i].n) && !(o == 2 && i == 3 && h_out == h0))
        return SANATAN_ERR_INVALID;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o].p, out[o].n, out[i].p, out[i].n)) return SANATAN_ERR_INVALID;
  }
  if (int s = check_arch()) return s;
  ScanArgs a;
  a.x = x;
  a.g = g;
  a.dtype = dtype;
  a.gate = gate;
  a.lens = lens;
  a.B = B;
  a.T = T;
  a.D = D;
  a.h0 = h0;
  a.y = y;
  a.h_out = h_out;
  a.marks = marks;
  return from_cuda(gated_scan_fwd_launch(a, static_cast<cudaStream_t>(stream)));
}

int sanatan_gated_scan_bwd(const void* x, const void* g, const void* dy, int dtype, int gate,
                           const int64_t* lens, int B, int T, int D, const float* marks,
                           const float* dh_out, void* dx, void* dg, float* dh0, void* stream) {
  if (int s = check_scan(dtype, gate, B, T, D)) return s;
  if (!ok_nullable(lens) || !ok_nullable(dh_out) || !ok_nullable(dh0)) return SANATAN_ERR_INVALID;
  if (static_cast<int64_t>(B) * D == 0) return SANATAN_OK;
  if (T > 0 && (!ok_ptr(x) || !ok_ptr(g) || dy == nullptr ||
                !at_element(dy, dtype == SANATAN_F32 ? 4 : 2) || !ok_ptr(marks) || !ok_ptr(dx) ||
                !ok_ptr(dg)))
    return SANATAN_ERR_INVALID;
  if (T == 0 && dh0 == nullptr) return SANATAN_OK;
  const size_t state = static_cast<size_t>(B) * D * 4;
  const size_t all = static_cast<size_t>(B) * T * D * (dtype == SANATAN_F32 ? 4 : 2);
  const size_t nm = sanatan_gated_scan_marks_size(B, T, D);
  const size_t len = static_cast<size_t>(B) * 8;
  const Range in[] = {{x, all}, {g, all}, {dy, all}, {lens, len}, {marks, nm}, {dh_out, state}};
  const Range out[] = {{dx, all}, {dg, all}, {dh0, state}};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 6; ++i)  // (dh0 may be dh_out)
      if (overlap(out[o].p, out[o].n, in[i].p, in[i].n) && !(o == 2 && i == 5 && dh0 == dh_out))
        return SANATAN_ERR_INVALID;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o].p, out[o].n, out[i].p, out[i].n)) return SANATAN_ERR_INVALID;
  }
  if (int s = check_arch()) return s;
  ScanBwdArgs a;
  a.x = x;
  a.g = g;
  a.dy = dy;
  a.dtype = dtype;
  a.gate = gate;
  a.lens = lens;
  a.B = B;
  a.T = T;
  a.D = D;
  a.marks = marks;
  a.dh_out = dh_out;
  a.dx = dx;
  a.dg = dg;
  a.dh0 = dh0;
  return from_cuda(gated_scan_bwd_launch(a, static_cast<cudaStream_t>(stream)));
}

int sanatan_gated_scan_step(float* h, const void* x, const void* g, int dtype, int gate, int N,
                            int D, void* y, void* stream) {
  if (int s = check_scan(dtype, gate, N, 1, D)) return s;
  const int64_t n = static_cast<int64_t>(N) * D;
  if (n == 0) return SANATAN_OK;
  if (!ok_floats(h) || !ok_ptr(x) || !ok_ptr(g) || !ok_ptr(y)) return SANATAN_ERR_INVALID;
  const size_t all = static_cast<size_t>(n) * (dtype == SANATAN_F32 ? 4 : 2);
  const size_t state = static_cast<size_t>(n) * 4;
  if (overlap(y, all, x, all) || overlap(y, all, g, all) || overlap(y, all, h, state) ||
      overlap(h, state, x, all) || overlap(h, state, g, all))
    return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  return from_cuda(gated_scan_step_launch(h, x, g, dtype, gate, n, y,
                                          static_cast<cudaStream_t>(stream)));
}

int sanatan_state_cache_write(const float* state, const float* exact, int layers, int B,
                              int64_t inner, int64_t exact_inner, const int64_t* pages,
                              int64_t num_pages, int fmt, void* codes, float* scales,
                              float* exact_cache, void* stream) {
  return state_cache(const_cast<float*>(state), const_cast<float*>(exact), layers, B, inner,
                     exact_inner, pages, num_pages, fmt, codes, scales, exact_cache, true, stream);
}

int sanatan_state_cache_read(const void* codes, const float* scales, const float* exact_cache,
                             int64_t num_pages, int fmt, const int64_t* pages, int layers, int B,
                             int64_t inner, int64_t exact_inner, float* state, float* exact,
                             void* stream) {
  return state_cache(state, exact, layers, B, inner, exact_inner, pages, num_pages, fmt,
                     const_cast<void*>(codes), const_cast<float*>(scales),
                     const_cast<float*>(exact_cache), false, stream);
}

int sanatan_layer_norm_fwd(const void* x, const void* residual, const float* weight,
                           const float* bias, int dtype, int64_t rows, int D, float eps, void* y,
                           void* sum, float* stats, void* stream) {
  if (int s = check_norm(dtype, rows, D)) return s;
  if (rows == 0 || D == 0) return SANATAN_OK;
  const size_t e = size_of(dtype), all = static_cast<size_t>(rows) * D * e;
  const size_t row = static_cast<size_t>(D) * 4;
  if (!at_elements({x, y}, e) || !at_elements({residual, sum}, e, true) ||
      !at_elements({weight, bias, stats}, 4, true))
    return SANATAN_ERR_INVALID;
  if (sum != nullptr && residual == nullptr) return SANATAN_ERR_INVALID;
  if (clash({{y, all}, {sum, all}, {stats, static_cast<size_t>(rows) * 8}},
            {{x, all}, {residual, all}, {weight, row}, {bias, row}}, {{1, 1}}))
    return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  NormArgs a;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.bias = bias;
  a.dtype = dtype;
  a.rows = rows;
  a.D = D;
  a.eps = eps;
  a.y = y;
  a.sum = sum;
  a.stats = stats;
  return from_cuda(layer_norm_fwd_launch(a, static_cast<cudaStream_t>(stream)));
}

size_t sanatan_layer_norm_bwd_workspace_size(int64_t rows, int D) {
  return layer_norm_bwd_workspace_bytes(rows, D);
}

int sanatan_layer_norm_bwd(const void* s, const float* weight, const void* dy, const void* ds,
                           const float* stats, int dtype, int64_t rows, int D, void* dx,
                           float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (int st = check_norm(dtype, rows, D)) return st;
  if (D == 0) return SANATAN_OK;
  const size_t e = size_of(dtype), all = static_cast<size_t>(rows) * D * e;
  const size_t row = static_cast<size_t>(D) * 4;
  if (!at_elements({weight, dweight, dbias, workspace}, 4, true)) return SANATAN_ERR_INVALID;
  if (rows > 0 && (!at_elements({s, dy, dx}, e) || !at_elements({ds}, e, true) ||
                   !at_elements({stats}, 4)))
    return SANATAN_ERR_INVALID;
  const bool sums = rows > 0 && (dweight != nullptr || dbias != nullptr);
  const size_t need = sums ? layer_norm_bwd_workspace_bytes(rows, D) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SANATAN_ERR_INVALID;
  if (clash({{dx, all}, {dweight, row}, {dbias, row}, {workspace, need}},
            {{s, all}, {weight, row}, {dy, all}, {ds, all}, {stats, static_cast<size_t>(rows) * 8}},
            {}))
    return SANATAN_ERR_INVALID;
  if (int st = check_arch()) return st;
  NormBwdArgs a;
  a.s = s;
  a.weight = weight;
  a.dy = dy;
  a.ds = ds;
  a.stats = stats;
  a.dtype = dtype;
  a.rows = rows;
  a.D = D;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.parts = static_cast<float*>(workspace);
  return from_cuda(layer_norm_bwd_launch(a, static_cast<cudaStream_t>(stream)));
}

int sanatan_causal_conv_fwd(const void* x, int64_t ldx, const float* w, const float* bias,
                            int dtype, int act, const int64_t* lens, int B, int T, int D, int K,
                            const float* s0, void* y, float* s_out, void* stream) {
  if (int s = check_conv(dtype, act, B, T, D, K, ldx)) return s;
  if (static_cast<int64_t>(B) * D == 0) return SANATAN_OK;
  const size_t e = size_of(dtype), state = static_cast<size_t>(B) * (K - 1) * D * 4;
  const int64_t tokens = static_cast<int64_t>(B) * T;
  if (!at_elements({w}, 4) || !at_elements({bias, s0, s_out}, 4, true) ||
      !at_elements({lens}, 8, true))
    return SANATAN_ERR_INVALID;
  if (T > 0 && !at_elements({x, y}, e)) return SANATAN_ERR_INVALID;
  if (clash({{y, span(tokens, D, D, e)}, {s_out, state}},
            {{x, span(tokens, ldx, D, e)},
             {w, static_cast<size_t>(D) * K * 4},
             {bias, static_cast<size_t>(D) * 4},
             {lens, static_cast<size_t>(B) * 8},
             {s0, state}}))
    return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  ConvArgs a;
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.bias = bias;
  a.dtype = dtype;
  a.act = act;
  a.lens = lens;
  a.B = B;
  a.T = T;
  a.D = D;
  a.K = K;
  a.s0 = s0;
  a.y = y;
  a.s_out = K > 1 ? s_out : nullptr;
  return from_cuda(causal_conv_fwd_launch(a, static_cast<cudaStream_t>(stream)));
}

size_t sanatan_causal_conv_bwd_workspace_size(int B, int T, int D, int K) {
  return causal_conv_bwd_workspace_bytes(B, T, D, K);
}

int sanatan_causal_conv_bwd(const void* x, int64_t ldx, const float* w, const float* bias,
                            const void* dy, int dtype, int act, const int64_t* lens, int B, int T,
                            int D, int K, const float* s0, const float* ds_out, void* dx,
                            float* dw, float* dbias, float* ds0, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (int s = check_conv(dtype, act, B, T, D, K, ldx)) return s;
  if (D == 0) return SANATAN_OK;
  const size_t e = size_of(dtype), state = static_cast<size_t>(B) * (K - 1) * D * 4;
  const int64_t tokens = static_cast<int64_t>(B) * T;
  if (!at_elements({w}, 4) || !at_elements({bias, s0, ds_out, dw, dbias, ds0, workspace}, 4, true) ||
      !at_elements({lens}, 8, true))
    return SANATAN_ERR_INVALID;
  if (tokens > 0 && !at_elements({x, dy, dx}, e)) return SANATAN_ERR_INVALID;
  const bool sums = dw != nullptr || dbias != nullptr;
  const size_t need = sums ? causal_conv_bwd_workspace_bytes(B, T, D, K) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SANATAN_ERR_INVALID;
  const size_t wide = static_cast<size_t>(D) * K * 4, row = static_cast<size_t>(D) * 4;
  if (clash({{dx, span(tokens, D, D, e)}, {dw, wide}, {dbias, row}, {ds0, state},
             {workspace, need}},
            {{x, span(tokens, ldx, D, e)}, {w, wide}, {bias, row}, {dy, span(tokens, D, D, e)},
             {lens, static_cast<size_t>(B) * 8}, {s0, state}, {ds_out, state}}))
    return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  ConvBwdArgs a;
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.bias = bias;
  a.dy = dy;
  a.dtype = dtype;
  a.act = act;
  a.lens = lens;
  a.B = B;
  a.T = T;
  a.D = D;
  a.K = K;
  a.s0 = s0;
  a.ds_out = ds_out;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.ds0 = ds0;
  a.parts = static_cast<float*>(workspace);
  return from_cuda(causal_conv_bwd_launch(a, static_cast<cudaStream_t>(stream)));
}

int sanatan_causal_conv_step(float* state, const void* x, int64_t ldx, const float* w,
                             const float* bias, int dtype, int act, int N, int D, int K, void* y,
                             void* stream) {
  if (int s = check_conv(dtype, act, N, 1, D, K, ldx)) return s;
  if (static_cast<int64_t>(N) * D == 0) return SANATAN_OK;
  const size_t e = size_of(dtype);
  if (!at_elements({x, y}, e) || !at_elements({w}, 4) || !at_elements({state}, 4, K == 1) ||
      !at_elements({bias}, 4, true))
    return SANATAN_ERR_INVALID;
  if (clash({{y, span(N, D, D, e)}, {state, static_cast<size_t>(N) * (K - 1) * D * 4}},
            {{x, span(N, ldx, D, e)}, {w, static_cast<size_t>(D) * K * 4},
             {bias, static_cast<size_t>(D) * 4}}))
    return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  ConvArgs a;
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.bias = bias;
  a.dtype = dtype;
  a.act = act;
  a.B = N;
  a.T = 1;
  a.D = D;
  a.K = K;
  a.y = y;
  a.s_out = state;
  return from_cuda(causal_conv_step_launch(a, static_cast<cudaStream_t>(stream)));
}

size_t sanatan_selective_scan_marks_size(int B, int T, int D, int N) {
  if (B < 0 || T < 0 || D < 0 || N < 0) return 0;
  return static_cast<size_t>(B) *
         ((static_cast<size_t>(T) + kSelectiveMark - 1) / kSelectiveMark) * D * N * sizeof(float);
}

size_t sanatan_selective_scan_fwd_workspace_size(int B, int T, int D, int N) {
  return N > kSelectiveStates ? 0 : selective_scan_fwd_workspace_bytes(B, T, D, N);
}

int sanatan_selective_scan_fwd(const void* u, const void* dt, const void* z, int64_t ldz,
                               const void* Bm, int64_t ldb, const void* Cm, int64_t ldc,
                               const float* A, const float* skip, const float* dt_bias, int dtype,
                               int softplus, const int64_t* lens, int B, int T, int D, int N,
                               const float* h0, void* y, float* h_out, float* marks,
                               void* workspace, size_t workspace_bytes, void* stream) {
  SelectiveArgs a;
  a.u = u;
  a.dt = dt;
  a.z = z;
  a.Bm = Bm;
  a.Cm = Cm;
  a.ldz = ldz;
  a.ldb = ldb;
  a.ldc = ldc;
  a.A = A;
  a.skip = skip;
  a.dt_bias = dt_bias;
  a.dtype = dtype;
  a.softplus = softplus != 0;
  a.lens = lens;
  a.B = B;
  a.T = T;
  a.D = D;
  a.N = N;
  a.h0 = h0;
  a.y = y;
  a.h_out = h_out;
  a.marks = marks;
  if (int s = check_selective(a)) return s;
  if (static_cast<int64_t>(B) * D == 0) return SANATAN_OK;
  const size_t e = size_of(dtype);
  const int64_t tokens = static_cast<int64_t>(B) * T;
  if (T > 0 && !at_elements({y}, e)) return SANATAN_ERR_INVALID;
  if (T == 0 && h_out == nullptr) return SANATAN_OK;
  const size_t need = selective_scan_fwd_workspace_bytes(B, T, D, N);
  if (need > 0 && (workspace == nullptr || !at_element(workspace, 4) || workspace_bytes < need))
    return SANATAN_ERR_INVALID;
  const size_t state = static_cast<size_t>(B) * D * N * 4, row = static_cast<size_t>(D) * 4;
  const size_t dense = span(tokens, D, D, e);
  if (clash({{y, dense}, {h_out, state}, {marks, sanatan_selective_scan_marks_size(B, T, D, N)},
             {workspace, need}},
            {{h0, state}, {u, dense}, {dt, dense}, {z, span(tokens, ldz, D, e)},
             {Bm, span(tokens, ldb, N, e)}, {Cm, span(tokens, ldc, N, e)},
             {A, static_cast<size_t>(D) * N * 4}, {skip, row}, {dt_bias, row},
             {lens, static_cast<size_t>(B) * 8}},
            {{1, 0}}))
    return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  return from_cuda(selective_scan_fwd_launch(a, workspace, static_cast<cudaStream_t>(stream)));
}

size_t sanatan_selective_scan_bwd_workspace_size(int B, int T, int D, int N) {
  return N > kSelectiveStates ? 0 : selective_scan_bwd_workspace_bytes(B, T, D, N);
}

int sanatan_selective_scan_bwd(const void* u, const void* dt, const void* z, int64_t ldz,
                               const void* Bm, int64_t ldb, const void* Cm, int64_t ldc,
                               const float* A, const float* skip, const float* dt_bias, int dtype,
                               int softplus, const int64_t* lens, int B, int T, int D, int N,
                               const void* dy, const float* marks, const float* dh_out, void* du,
                               void* ddt, void* dz, float* dA, void* dB, void* dC, float* dskip,
                               float* ddt_bias, float* dh0, void* workspace,
                               size_t workspace_bytes, void* stream) {
  SelectiveBwdArgs args;
  SelectiveArgs& a = args.f;
  a.u = u;
  a.dt = dt;
  a.z = z;
  a.Bm = Bm;
  a.Cm = Cm;
  a.ldz = ldz;
  a.ldb = ldb;
  a.ldc = ldc;
  a.A = A;
  a.skip = skip;
  a.dt_bias = dt_bias;
  a.dtype = dtype;
  a.softplus = softplus != 0;
  a.lens = lens;
  a.B = B;
  a.T = T;
  a.D = D;
  a.N = N;
  if (int s = check_selective(a)) return s;
  const size_t e = size_of(dtype);
  const int64_t tokens = static_cast<int64_t>(B) * T;
  args.dB = dB;
  args.dC = dC;
  if (D == 0) {  // (dB and dC are sums over no channels)
    const size_t pair = span(tokens, N, N, e);
    if (pair == 0) return SANATAN_OK;
    if (!at_elements({dB, dC}, e)) return SANATAN_ERR_INVALID;
    if (clash({{dB, pair}, {dC, pair}}, {{Bm, span(tokens, ldb, N, e)},
                                         {Cm, span(tokens, ldc, N, e)},
                                         {lens, static_cast<size_t>(B) * 8}}))
      return SANATAN_ERR_INVALID;
    if (int s = check_arch()) return s;
    return from_cuda(selective_scan_bwd_launch(args, nullptr, static_cast<cudaStream_t>(stream)));
  }
  if (!at_elements({dA}, 4) || !at_elements({dskip, ddt_bias, dh0, dh_out}, 4, true))
    return SANATAN_ERR_INVALID;
  if (tokens > 0 && (!at_elements({dy, du, ddt, dB, dC}, e) || !at_elements({dz}, e, z == nullptr) ||
                !at_elements({marks}, 4)))
    return SANATAN_ERR_INVALID;
  if (z == nullptr && dz != nullptr) return SANATAN_ERR_INVALID;
  const size_t need = selective_scan_bwd_workspace_bytes(B, T, D, N);
  if (need > 0 && (workspace == nullptr || !at_element(workspace, 4) || workspace_bytes < need))
    return SANATAN_ERR_INVALID;
  const size_t state = static_cast<size_t>(B) * D * N * 4, row = static_cast<size_t>(D) * 4;
  const size_t dense = span(tokens, D, D, e), pair = span(tokens, N, N, e);
  const size_t matrix = static_cast<size_t>(D) * N * 4;
  if (clash({{dh0, state}, {du, dense}, {ddt, dense}, {dz, dense}, {dA, matrix}, {dB, pair},
             {dC, pair}, {dskip, row}, {ddt_bias, row}, {workspace, need}},
            {{dh_out, state}, {u, dense}, {dt, dense}, {z, span(tokens, ldz, D, e)},
             {Bm, span(tokens, ldb, N, e)}, {Cm, span(tokens, ldc, N, e)}, {A, matrix},
             {skip, row}, {dt_bias, row}, {lens, static_cast<size_t>(B) * 8}, {dy, dense},
             {marks, sanatan_selective_scan_marks_size(B, T, D, N)}},
            {{0, 0}}))
    return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  args.dy = dy;
  args.marks = marks;
  args.dh_out = dh_out;
  args.du = du;
  args.ddt = ddt;
  args.dz = dz;
  args.dA = dA;
  args.dskip = dskip;
  args.ddt_bias = ddt_bias;
  args.dh0 = dh0;
  return from_cuda(selective_scan_bwd_launch(args, workspace, static_cast<cudaStream_t>(stream)));
}

int sanatan_selective_scan_step(float* h, const void* u, const void* dt, const void* z,
                                int64_t ldz, const void* Bm, int64_t ldb, const void* Cm,
                                int64_t ldc, const float* A, const float* skip,
                                const float* dt_bias, int dtype, int softplus, int nseq, int D,
                                int N, void* y, void* stream) {
  SelectiveArgs a;
  a.u = u;
  a.dt = dt;
  a.z = z;
  a.Bm = Bm;
  a.Cm = Cm;
  a.ldz = ldz;
  a.ldb = ldb;
  a.ldc = ldc;
  a.A = A;
  a.skip = skip;
  a.dt_bias = dt_bias;
  a.dtype = dtype;
  a.softplus = softplus != 0;
  a.B = nseq;
  a.T = 1;
  a.D = D;
  a.N = N;
  a.y = y;
  a.h_out = h;
  if (int s = check_selective(a)) return s;
  if (static_cast<int64_t>(nseq) * D == 0) return SANATAN_OK;
  const size_t e = size_of(dtype), row = static_cast<size_t>(D) * 4, dense = span(nseq, D, D, e);
  if (!at_elements({h}, 4) || !at_elements({y}, e)) return SANATAN_ERR_INVALID;
  if (clash({{y, dense}, {h, static_cast<size_t>(nseq) * D * N * 4}},
            {{u, dense}, {dt, dense}, {z, span(nseq, ldz, D, e)}, {Bm, span(nseq, ldb, N, e)},
             {Cm, span(nseq, ldc, N, e)}, {A, row * N}, {skip, row}, {dt_bias, row}}))
    return SANATAN_ERR_INVALID;
  if (int s = check_arch()) return s;
  return from_cuda(selective_scan_step_launch(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
