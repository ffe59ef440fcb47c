// Internal launch interfaces between the C ABI (api.cu) and the kernels.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "sanatan.h"

namespace sanatan {

struct ChunkFwdArgs {
  const void* q;
  const void* k;
  const void* v;
  int in_dtype;
  const float* gamma;
  const float* omega;
  const float* phi;
  int B, H, T, d, dv;
  int64_t pos0;
  float eps;
  const float* S0;
  const float* z0;
  float* o;
  float* D;
  float* S_out;
  float* z_out;
  void* workspace;
  size_t workspace_bytes;
};

struct ChunkBwdArgs {
  ChunkFwdArgs f;
  const float* o;
  const float* Dn;
  const void* dO;
  int grad_dtype;
  void* dq;
  void* dk;
  void* dv;
  float* dgamma;
  float* domega;
  float* dphi;
  void* workspace;
  size_t workspace_bytes;
  const void* fwd_workspace;   // the forward's workspace (its per-segment sums) or null
  size_t fwd_workspace_bytes;
};

// Events recorded around the dominant kernel of a chunk_fwd / chunk_bwd call
// (bench instrumentation; null when unused).
struct ProfileEvents {
  cudaEvent_t start = nullptr;
  cudaEvent_t stop = nullptr;
};
ProfileEvents& profile_events();

cudaError_t featurize_launch(const void* u, int u_dtype, const float* gamma, const float* omega,
                             const float* phi, int B, int H, int T, int d, int64_t pos0,
                             void* out, int out_dtype, cudaStream_t st);

// phi = scale tanh(raw) (dphi == null) or dphi scale (1 - tanh^2(raw)).
cudaError_t rate_launch(const float* raw, const float* dphi, int n, float scale, float* out,
                        cudaStream_t st);

cudaError_t decode_step_launch(float* S, float* z, const float* q, const float* k,
                               const float* v, const float* gamma, const float* omega,
                               const float* phi, const int64_t* pos, int N, int G, float eps,
                               float* o, cudaStream_t st);

// Harmonic feature map (harmonics n = 1..N, N <= 3).
struct HarmonicFeatArgs {
  const void* u;
  int u_dtype;
  const float* gamma;
  const float* omega;
  const float* phi;
  int B, H, T;
  int64_t pos0;
  int harmonics;
  void* out;
  int out_dtype;
};
cudaError_t featurize_harmonic_launch(const HarmonicFeatArgs& a, cudaStream_t st);
// f32 chunked forward with the harmonic map (N <= 3; bf16 or f32 loads).
cudaError_t chunk_fwd_harmonic_launch(const ChunkFwdArgs& a, int harmonics, cudaStream_t st);
// Its backward (N <= 3); the workspace holds dN and dD (none for N = 1).
size_t chunk_bwd_harmonic_workspace_bytes(int B, int H, int T, int harmonics);
cudaError_t chunk_bwd_harmonic_launch(const ChunkBwdArgs& a, int harmonics, cudaStream_t st);
cudaError_t decode_harmonic_launch(float* S, float* z, const float* q, const float* k,
                                   const float* v, const float* gamma, const float* omega,
                                   const float* phi, const int64_t* pos, int N, int G, float eps,
                                   int harmonics, float* o, cudaStream_t st);

// One token through L attention layers (stack.cu): one cooperative launch.
struct StackArgs {
  float* x;              // [B, heads * 64], updated in place
  const float* Wqkv;     // [L, heads * 64, 3 * heads * 64]
  const float* Wo;       // [L, heads * 64, heads * 64]
  float* S;              // [L, B * heads, 384, 64]
  float* z;              // [L, B * heads, 384]
  const float* gamma;    // [L, heads]
  const float* omega;    // [L, heads, 64]
  const float* phi;      // [L, heads, 64]
  const int64_t* pos;    // [B * heads]
  int B, L, heads;
  float eps;
  void* workspace;       // stack_workspace_bytes
};
size_t stack_workspace_bytes(int B, int heads, int d);
int stack_max_batch();
cudaError_t stack_decode_launch(const StackArgs& a, cudaStream_t st);
int stack_read_and_clear_error(cudaStream_t st);

size_t chunk_fwd_simt_smem_bytes();
size_t chunk_bwd_simt_smem_bytes();
cudaError_t chunk_bwd_simt_launch(const ChunkBwdArgs& a, cudaStream_t st);
cudaError_t chunk_fwd_simt_launch(const ChunkFwdArgs& a, cudaStream_t st);

}  // namespace sanatan

namespace sanatan {
int tc_segments(int B, int H, int T);
size_t chunk_fwd_tc_workspace_bytes(int B, int H, int T);
cudaError_t chunk_fwd_tc_launch(const ChunkFwdArgs& a, cudaStream_t st);
int tc_read_and_clear_error(cudaStream_t st);
// One CTA whose bounded wait on an mbarrier nobody arrives at (unless
// `arrive`) gives up after timeout_ns and records a timeout.
cudaError_t tc_timeout_probe_launch(uint64_t timeout_ns, int arrive, cudaStream_t st);

// One causal (or, reversed, anti-causal) attention on the tensor-core kernel,
// bf16 q, k, v of shape [B, H, T, 64].  `extra` replaces the ones column of
// [V | 1] (the denominator) by a per-token value; `deltas` is the workspace of
// per-segment state sums, B * H * tc_segments * 321 * 80 floats.
struct TcJob {
  const void* q = nullptr;
  const void* k = nullptr;
  const void* v = nullptr;
  const float* extra = nullptr;
  const float* gamma = nullptr;
  const float* omega = nullptr;
  const float* phi = nullptr;
  int B = 0, H = 0, T = 0;
  int64_t pos0 = 0;
  float eps = 0.f;
  const float* S0 = nullptr;
  const float* z0 = nullptr;
  void* o = nullptr;        // f32 or (out_bf16) bf16 [B, H, T, 64]
  float* Dn = nullptr;
  float* S_out = nullptr;
  float* z_out = nullptr;
  int reverse = 0;          // row u is processed at position T-1-u
  int normalize = 1;        // 0: write the numerator only
  int out_bf16 = 0;
  float* deltas = nullptr;
  int deltas_ready = 0;     // the state-only pass has already filled `deltas`
  int record_events = 1;    // bracket the main launch with the profile events
  int nseg = 0;             // segments per sequence (0: tc_segments)
};
// State-only pass: the sums of every segment but the last into job.deltas.
cudaError_t tc_state_pass(const TcJob& job, cudaStream_t st);
// The attention itself (running the state-only pass first unless deltas_ready).
cudaError_t tc_attention(const TcJob& job, cudaStream_t st);

size_t chunk_bwd_tc_workspace_bytes(int B, int H, int T);
// Segments that a workspace of `bytes` holds (at most tc_segments; 1 needs none).
int tc_segments_fit(int B, int H, int T, size_t bytes);
int chunk_fwd_checked(const void* q, const void* k, const void* v, int in_dtype,
                      const float* gamma, const float* omega, const float* phi, int B, int H,
                      int T, int d, int dv, int64_t pos0, float eps, const float* S0,
                      const float* z0, float* o, float* D, float* S_out, float* z_out,
                      void* workspace, size_t workspace_bytes, void* stream, bool fewer_segments);
cudaError_t chunk_bwd_tc_launch(const ChunkBwdArgs& a, cudaStream_t st);
int bwd_tc_read_and_clear_error(cudaStream_t st);

// Power-sharpened causal attention (bf16 q, k, v [B, H, T, 64], integer p).
struct PowFwdArgs {
  const void* q = nullptr;
  const void* k = nullptr;
  const void* v = nullptr;
  const float* gamma = nullptr;
  const float* omega = nullptr;
  const float* phi = nullptr;
  int B = 0, H = 0, T = 0;
  int64_t pos0 = 0;
  int p = 1;
  float eps = 0.f;
  float* o = nullptr;
  float* D = nullptr;
  void* workspace = nullptr;   // pow_fwd_tc_workspace_bytes
};
size_t pow_fwd_tc_workspace_bytes(int B, int H, int T);
cudaError_t pow_fwd_tc_launch(const PowFwdArgs& a, cudaStream_t st);
// The four- (channels = 4) or three-channel (channels = 3, with `shift`) map in
// the same kernels; p in {1, 2, 4}.
cudaError_t ablation_fwd_tc_launch(const PowFwdArgs& a, int channels, float shift,
                                   cudaStream_t st);
// The preparation kernel alone (features and [V | 1 | 0] into a.workspace).
cudaError_t pow_prep_launch(const PowFwdArgs& a, cudaStream_t st);

// Gradients of the power-sharpened attention.
struct PowBwdArgs {
  PowFwdArgs f;               // q, k, v, params, sizes, p, eps; f.workspace = the whole workspace
  const float* o = nullptr;   // [B, H, T, 64] f32, the forward's output
  const float* D = nullptr;   // [B, H, T] f32, the forward's denominator (without eps)
  const void* dO = nullptr;   // [B, H, T, 64], grad_dtype
  int grad_dtype = 0;
  void* dq = nullptr;         // bf16 [B, H, T, 64]
  void* dk = nullptr;
  void* dv = nullptr;
  float* dgamma = nullptr;    // [H], overwritten
  float* domega = nullptr;    // [H, 64], overwritten
  float* dphi = nullptr;      // [H, 64], overwritten (may be null)
};
size_t pow_bwd_tc_workspace_bytes(int B, int H, int T);
cudaError_t pow_bwd_tc_launch(const PowBwdArgs& a, cudaStream_t st);
int pow_bwd_tc_read_and_clear_error(cudaStream_t st);
int pow_tc_read_and_clear_error(cudaStream_t st);

// Gated linear recurrence over [B, T, D] (gated_scan_fwd.cu, gated_scan_bwd.cu).
constexpr int kScanMark = 64;  // tokens between two marks (saved states)
struct ScanArgs {
  const void* x = nullptr;
  const void* g = nullptr;
  int dtype = 0, gate = 0;
  const int64_t* lens = nullptr;  // [B] or null
  int B = 0, T = 0, D = 0;
  const float* h0 = nullptr;      // [B, D] or null
  void* y = nullptr;
  float* h_out = nullptr;         // [B, D] or null
  float* marks = nullptr;         // [B, ceil(T / 64), D] or null
};
struct ScanBwdArgs {
  const void* x = nullptr;
  const void* g = nullptr;
  const void* dy = nullptr;
  int dtype = 0, gate = 0;
  const int64_t* lens = nullptr;
  int B = 0, T = 0, D = 0;
  const float* marks = nullptr;
  const float* dh_out = nullptr;  // [B, D] or null
  void* dx = nullptr;
  void* dg = nullptr;
  float* dh0 = nullptr;           // [B, D] or null
};
cudaError_t gated_scan_fwd_launch(const ScanArgs& a, cudaStream_t st);
int scan_fwd_read_and_clear_error(cudaStream_t st);
int scan_bwd_read_and_clear_error(cudaStream_t st);
cudaError_t gated_scan_bwd_launch(const ScanBwdArgs& a, cudaStream_t st);
cudaError_t gated_scan_step_launch(float* h, const void* x, const void* g, int dtype, int gate,
                                   int64_t n, void* y, cudaStream_t st);

// Quantised state cache (state_cache.cu).
struct CacheArgs {
  float* state = nullptr;         // [layers, B, inner]
  float* exact = nullptr;         // [layers, B, exact_inner] or null
  int layers = 0, B = 0;
  int64_t inner = 0, exact_inner = 0;
  const int64_t* pages = nullptr;  // [B]
  int64_t num_pages = 0;
  int fmt = 0;
  void* codes = nullptr;           // [num_pages, layers, ceil(inner / 64), 64]
  float* scales = nullptr;         // [num_pages, layers, ceil(inner / 64)]
  float* exact_cache = nullptr;    // [num_pages, layers, exact_inner] or null
  unsigned blocks = 0;             // thread blocks of one stretch
  int begin = 0, end = 0;          // sequences of one launch (set by the launcher)
};
int64_t state_cache_blocks(int64_t inner);
cudaError_t state_cache_launch(CacheArgs a, bool write, cudaStream_t st);

constexpr int kSms = 152;  // of a GB300, for the plans of the layers below

// Layer norm of rows of D values (layer_norm.cu).
constexpr int kNormParts = 304;    // partial sums of dw and db: blocks of the backward at most
struct NormArgs {
  const void* x = nullptr;
  const void* residual = nullptr;  // or null
  const float* weight = nullptr;   // [D] or null (1)
  const float* bias = nullptr;     // [D] or null (0)
  int dtype = 0, D = 0;
  int64_t rows = 0;
  float eps = 0.f;
  void* y = nullptr;
  void* sum = nullptr;             // x + residual or null
  float* stats = nullptr;          // [rows, 2] mean, 1 / sqrt(var + eps), or null
};
struct NormBwdArgs {
  const void* s = nullptr;         // what was normalised
  const float* weight = nullptr;
  const void* dy = nullptr;
  const void* ds = nullptr;        // or null
  const float* stats = nullptr;
  int dtype = 0, D = 0;
  int64_t rows = 0;
  void* dx = nullptr;
  float* dweight = nullptr;        // [D] or null
  float* dbias = nullptr;          // [D] or null
  float* parts = nullptr;          // layer_norm_bwd_workspace_bytes
};
size_t layer_norm_bwd_workspace_bytes(int64_t rows, int D);
cudaError_t layer_norm_fwd_launch(const NormArgs& a, cudaStream_t st);
cudaError_t layer_norm_bwd_launch(const NormBwdArgs& a, cudaStream_t st);

// Short causal convolution over [B, T, D] (causal_conv.cu).
constexpr int kConvTaps = 8;    // K at most
constexpr int kConvParts = 256; // partial sums of dw and dbias at most
struct ConvArgs {
  const void* x = nullptr;
  int64_t ldx = 0;                 // values between two tokens of x
  const float* w = nullptr;        // [D, K]
  const float* bias = nullptr;     // [D] or null
  int dtype = 0, act = 0;
  const int64_t* lens = nullptr;   // [B] or null
  int B = 0, T = 0, D = 0, K = 0;
  const float* s0 = nullptr;       // [B, K - 1, D] or null
  void* y = nullptr;
  float* s_out = nullptr;          // [B, K - 1, D] or null (the step's state)
  int run = 0, runs = 0;           // tokens of a run, runs of a sequence (set by the launcher)
};
struct ConvBwdArgs {
  const void* x = nullptr;
  int64_t ldx = 0;
  const float* w = nullptr;
  const float* bias = nullptr;
  const void* dy = nullptr;
  int dtype = 0, act = 0;
  const int64_t* lens = nullptr;
  int B = 0, T = 0, D = 0, K = 0;
  const float* s0 = nullptr;
  const float* ds_out = nullptr;   // [B, K - 1, D] or null
  void* dx = nullptr;
  float* dw = nullptr;             // [D, K] or null
  float* dbias = nullptr;          // [D] or null
  float* ds0 = nullptr;            // [B, K - 1, D] or null
  float* parts = nullptr;          // causal_conv_bwd_workspace_bytes
  int run = 0, runs = 0;
};
size_t causal_conv_bwd_workspace_bytes(int B, int T, int D, int K);
cudaError_t causal_conv_fwd_launch(const ConvArgs& a, cudaStream_t st);
cudaError_t causal_conv_bwd_launch(const ConvBwdArgs& a, cudaStream_t st);
cudaError_t causal_conv_step_launch(const ConvArgs& a, cudaStream_t st);

// Selective state space scan over [B, T, D] with N states a channel (selective_scan_fwd.cu,
// selective_scan_bwd.cu).
constexpr int kSelectiveMark = 16;      // tokens between two marks (saved states)
constexpr int kSelectiveStates = 128;   // N at most
struct SelectiveArgs {
  const void* u = nullptr;
  const void* dt = nullptr;
  const void* z = nullptr;          // or null
  const void* Bm = nullptr;
  const void* Cm = nullptr;
  int64_t ldz = 0, ldb = 0, ldc = 0;  // values between two tokens
  const float* A = nullptr;         // [D, N]
  const float* skip = nullptr;      // [D] or null
  const float* dt_bias = nullptr;   // [D] or null
  int dtype = 0, softplus = 0;
  const int64_t* lens = nullptr;    // [B] or null
  int B = 0, T = 0, D = 0, N = 0;
  const float* h0 = nullptr;        // [B, D, N] or null
  void* y = nullptr;
  float* h_out = nullptr;           // [B, D, N] or null (the step's state)
  float* marks = nullptr;           // [B, ceil(T / 16), D, N] or null
  // set by the launchers
  bool vec = false;                 // states are read and written four at a time
  int blocks = 0, segments = 1, tiles_per_segment = 0;  // of channels; of tokens
  float* carry = nullptr;           // [B, segments, D, N]
  float* sums = nullptr;            // [B, segments, D]
};
int selective_lanes(int N);
int selective_blocks(int D, int N);
int selective_segments(int B, int T, int D, int N, int* tiles_per_segment);
size_t selective_scan_fwd_workspace_bytes(int B, int T, int D, int N);
cudaError_t selective_scan_fwd_launch(SelectiveArgs a, void* workspace, cudaStream_t st);
cudaError_t selective_scan_step_launch(SelectiveArgs a, cudaStream_t st);

struct SelectiveBwdArgs {
  SelectiveArgs f;                  // inputs, sizes and plan (y, h0, h_out, f.marks: unused)
  const void* dy = nullptr;
  const float* marks = nullptr;
  const float* dh_out = nullptr;    // [B, D, N] or null
  void* du = nullptr;
  void* ddt = nullptr;
  void* dz = nullptr;               // where there is a z
  float* dA = nullptr;
  void* dB = nullptr;
  void* dC = nullptr;
  float* dskip = nullptr;           // [D] or null
  float* ddt_bias = nullptr;        // [D] or null
  float* dh0 = nullptr;             // [B, D, N] or null
  // set by the launcher
  int pieces = 1, piece = 0;        // of a segment, walked one after the other from the last
  int tiles_per_piece = 0;
  // parts in the workspace
  float* pairs = nullptr;           // dB, dC: [blocks of channels, B, T, 2, N], or of a
                                    // piece: [.., B, segments, tiles_per_piece * 16, 2, N]
  float* params = nullptr;          // [B, segments, D, N]: dA
  float* channels = nullptr;        // [B, segments, 2, D]: dskip, ddt_bias
  float* lanes = nullptr;           // [B, segments, 2, 16, D]: theirs, between two pieces
};
size_t selective_scan_bwd_workspace_bytes(int B, int T, int D, int N);
cudaError_t selective_scan_bwd_launch(SelectiveBwdArgs a, void* workspace, cudaStream_t st);
}  // namespace sanatan
