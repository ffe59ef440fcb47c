"""Thin ctypes binding of libsanatan.so (C ABI declared in include/sanatan.h).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current CUDA
stream.  The library is loaded on first use; if it has not been built, every
call raises RuntimeError (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch
from torch.autograd.function import once_differentiable

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libsanatan.so")

SANATAN_F32 = 0
SANATAN_BF16 = 1
_DT = {torch.float32: SANATAN_F32, torch.bfloat16: SANATAN_BF16}
_FLOATS = (torch.float32, torch.bfloat16)

_c_int, _c_i64, _c_f, _c_sz, _c_p = (ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                     ctypes.c_size_t, ctypes.c_void_p)

_SIGS = {
    "sanatan_status_string": (ctypes.c_char_p, [_c_int]),
    "sanatan_abi_version": (_c_int, []),
    "sanatan_state_bytes": (_c_sz, [_c_int] * 4),
    "sanatan_featurize": (_c_int, [_c_p, _c_int, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_int,
                                   _c_i64, _c_p, _c_int, _c_p]),
    "sanatan_rate_from_raw": (_c_int, [_c_p, _c_int, _c_f, _c_p, _c_p]),
    "sanatan_rate_from_raw_bwd": (_c_int, [_c_p, _c_p, _c_int, _c_f, _c_p, _c_p]),
    "sanatan_eps_raw": (_c_f, [_c_f, _c_int, _c_int]),
    "sanatan_chunk_fwd_workspace_size": (_c_sz, [_c_int] * 6),
    "sanatan_chunk_fwd_plan": (_c_int, [_c_int] * 5 + [_c_p, _c_p]),
    "sanatan_chunk_fwd": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_int, _c_int,
                                   _c_int, _c_int, _c_int, _c_i64, _c_f, _c_p, _c_p, _c_p, _c_p,
                                   _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sanatan_chunk_fwd_noalloc_max_scratch_bytes": (_c_sz, []),
    "sanatan_chunk_fwd_noalloc": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int,
                                           _c_int, _c_int, _c_int, _c_i64, _c_f, _c_p, _c_p, _c_p,
                                           _c_p, _c_p, _c_p, _c_p]),
    "sanatan_chunk_bwd_workspace_size": (_c_sz, [_c_int] * 6),
    "sanatan_chunk_bwd": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_int, _c_int,
                                   _c_int, _c_int, _c_int, _c_i64, _c_f, _c_p, _c_p, _c_p, _c_p,
                                   _c_p, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz,
                                   _c_p]),
    "sanatan_power_fwd_workspace_size": (_c_sz, [_c_int] * 5),
    "sanatan_power_fwd": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int,
                                   _c_int, _c_int, _c_i64, _c_int, _c_f, _c_p, _c_p, _c_p, _c_sz,
                                   _c_p]),
    "sanatan_ablation_fwd": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int,
                                      _c_int, _c_int, _c_i64, _c_int, _c_int, _c_f, _c_f, _c_p,
                                      _c_p, _c_p, _c_sz, _c_p]),
    "sanatan_power_bwd_workspace_size": (_c_sz, [_c_int] * 5),
    "sanatan_power_bwd": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int,
                                   _c_int, _c_int, _c_i64, _c_int, _c_f, _c_p, _c_p, _c_p, _c_int,
                                   _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sanatan_device_status": (_c_int, [_c_p]),
    "sanatan_set_profile_events": (_c_int, [_c_p, _c_p]),
    "sanatan_selftest_wait_timeout": (_c_int, [ctypes.c_uint64, _c_int, _c_p]),
    "sanatan_stack_decode_workspace_size": (_c_sz, [_c_int] * 3),
    "sanatan_stack_decode_step": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                           _c_int, _c_int, _c_int, _c_int, _c_f, _c_p, _c_sz,
                                           _c_p]),
    "sanatan_state_bytes_harmonic": (_c_sz, [_c_int] * 5),
    "sanatan_featurize_harmonic": (_c_int, [_c_p, _c_int, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int,
                                            _c_int, _c_i64, _c_int, _c_p, _c_int, _c_p]),
    "sanatan_chunk_fwd_harmonic": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_int,
                                            _c_int, _c_int, _c_int, _c_int, _c_i64, _c_int, _c_f,
                                            _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "sanatan_chunk_bwd_harmonic_workspace_size": (_c_sz, [_c_int] * 6),
    "sanatan_chunk_bwd_harmonic": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_int,
                                            _c_int, _c_int, _c_int, _c_int, _c_i64, _c_int, _c_f,
                                            _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p,
                                            _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sanatan_decode_step_harmonic": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                              _c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_f,
                                              _c_p, _c_p]),
    "sanatan_decode_step": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int,
                                     _c_int, _c_int, _c_int, _c_f, _c_p, _c_p]),
    "sanatan_gated_scan_marks_size": (_c_sz, [_c_int] * 3),
    "sanatan_gated_scan_fwd": (_c_int, [_c_p, _c_p, _c_int, _c_int, _c_p, _c_int, _c_int, _c_int,
                                        _c_p, _c_p, _c_p, _c_p, _c_p]),
    "sanatan_gated_scan_bwd": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_int, _c_p, _c_int, _c_int,
                                        _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "sanatan_gated_scan_step": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_p,
                                         _c_p]),
    "sanatan_state_cache_write": (_c_int, [_c_p, _c_p, _c_int, _c_int, _c_i64, _c_i64, _c_p,
                                           _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p]),
    "sanatan_state_cache_read": (_c_int, [_c_p, _c_p, _c_p, _c_i64, _c_int, _c_p, _c_int, _c_int,
                                          _c_i64, _c_i64, _c_p, _c_p, _c_p]),
}

_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """The loaded library with argument types set (raises if not built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"{LIB_PATH} is missing: build it with "
                        "`python -m constant_state_recurrence_gb300.build` (there is no fallback)")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in _SIGS.items():
                    fn = getattr(handle, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = handle
    return _lib


def exported_symbols():
    return list(_SIGS)


class SanatanError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = lib().sanatan_status_string(status).decode()
        super().__init__(f"{fn} failed with status {status}: {msg}")


def _check(fn, status):
    if status != 0:
        raise SanatanError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t, name, dtypes=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _need_params(gamma, omega, phi, H, d):
    """gamma [H], omega [H, d], phi [H, d] float32 on the device (the kernels
    read H rows of each)."""
    _need(gamma, "gamma", (torch.float32,), (H,))
    _need(omega, "omega", (torch.float32,), (H, d))
    _need(phi, "phi", (torch.float32,), (H, d))


def device_status(device=None):
    """Synchronise the current stream and raise if a kernel of the library gave
    up a bounded device-side wait since the last check."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _check("sanatan_device_status", lib().sanatan_device_status(_stream(dev)))


def selftest_wait_timeout(timeout_ns=1_000_000, arrive=False, device=None):
    """Enqueue the library's failure-detection probe: a bounded wait on an
    mbarrier nobody arrives at (or, with arrive=True, one that completes)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _check("sanatan_selftest_wait_timeout",
           lib().sanatan_selftest_wait_timeout(int(timeout_ns), int(bool(arrive)), _stream(dev)))


def set_profile_events(start=None, stop=None):
    """Record torch.cuda.Event `start`/`stop` around the dominant kernel of the
    following chunk_fwd / chunk_bwd calls of this thread (None, None: off)."""
    for ev in (start, stop):
        if ev is not None and ev.cuda_event == 0:
            ev.record()  # torch creates the CUDA event lazily, on first record
    a = None if start is None else ctypes.c_void_p(start.cuda_event)
    b = None if stop is None else ctypes.c_void_p(stop.cuda_event)
    _check("sanatan_set_profile_events", lib().sanatan_set_profile_events(a, b))


def state_bytes(layers, heads, d=64, dv=64):
    return int(lib().sanatan_state_bytes(layers, heads, d, dv))


def sanatan_featurize(u, gamma, omega, phi, pos0=0, out_dtype=None, out=None):
    """Phi(u) [B, H, T, 6d] (index 6a + c) for u [B, H, T, d]."""
    _need(u, "u", (torch.float32, torch.bfloat16))
    B, H, T, d = u.shape
    odt = out_dtype or torch.float32
    if out is None:
        out = torch.empty(B, H, T, 6 * d, dtype=odt, device=u.device)
    _need(out, "out", (torch.float32, torch.bfloat16), (B, H, T, 6 * d))
    _need_params(gamma, omega, phi, H, d)
    st = lib().sanatan_featurize(_ptr(u), _DT[u.dtype], _ptr(gamma), _ptr(omega), _ptr(phi),
                                 B, H, T, d, int(pos0), _ptr(out), _DT[out.dtype],
                                 _stream(u.device))
    _check("sanatan_featurize", st)
    return out


RATE_SCALE = 0.01   # the pages' lambda = 0.01 tanh(lambda_raw)


def rate_from_raw(lambda_raw, scale=RATE_SCALE, out=None):
    """phi = scale * tanh(lambda_raw) (float32, on the device)."""
    _need(lambda_raw, "lambda_raw", (torch.float32,))
    out = torch.empty_like(lambda_raw) if out is None else out
    _need(out, "phi", (torch.float32,), tuple(lambda_raw.shape))
    _check("sanatan_rate_from_raw",
           lib().sanatan_rate_from_raw(_ptr(lambda_raw), lambda_raw.numel(), float(scale),
                                       _ptr(out), _stream(lambda_raw.device)))
    return out


def rate_from_raw_bwd(lambda_raw, dphi, scale=RATE_SCALE, out=None):
    """dlambda_raw = dphi * scale * (1 - tanh^2(lambda_raw))."""
    _need(lambda_raw, "lambda_raw", (torch.float32,))
    _need(dphi, "dphi", (torch.float32,), tuple(lambda_raw.shape))
    out = torch.empty_like(lambda_raw) if out is None else out
    _check("sanatan_rate_from_raw_bwd",
           lib().sanatan_rate_from_raw_bwd(_ptr(lambda_raw), _ptr(dphi), lambda_raw.numel(),
                                           float(scale), _ptr(out), _stream(lambda_raw.device)))
    return out


def eps_raw(eps, d=64, convention=0):
    """c * eps with c = 4d + 1e-6 (convention 0) or 4d * 1e-6 (convention 1)."""
    return float(lib().sanatan_eps_raw(float(eps), int(d), int(convention)))


def chunk_fwd_workspace_size(B, H, T, d=64, dv=64, dtype=torch.bfloat16):
    return int(lib().sanatan_chunk_fwd_workspace_size(B, H, T, d, dv, _DT[dtype]))


def chunk_fwd_plan(B, H, T, dtype=torch.bfloat16, has_initial_state=False):
    """(segments per sequence, kernel launches per call) of sanatan_chunk_fwd."""
    seg, nl = ctypes.c_int(0), ctypes.c_int(0)
    _check("sanatan_chunk_fwd_plan",
           lib().sanatan_chunk_fwd_plan(B, H, T, _DT[dtype], int(bool(has_initial_state)),
                                        ctypes.byref(seg), ctypes.byref(nl)))
    return seg.value, nl.value


def sanatan_chunk_fwd(q, k, v, gamma, omega, phi, pos0=0, eps=0.0, S0=None, z0=None,
                      want_D=True, want_state=False, out=None, D_out=None, workspace=None):
    """Causal p=1 attention over [B, H, T] sequences.

    Returns (o [B,H,T,dv] f32, D [B,H,T] f32 or None, S [B,H,6d,dv] or None,
    z [B,H,6d] or None)."""
    _need(q, "q", (torch.float32, torch.bfloat16))
    B, H, T, d = q.shape
    _need(k, "k", (q.dtype,), (B, H, T, d))
    _need(v, "v", (q.dtype,))
    dv = v.shape[-1]
    _need(v, "v", (q.dtype,), (B, H, T, dv))
    _need_params(gamma, omega, phi, H, d)
    dev = q.device
    F = 6 * d
    o = out if out is not None else torch.empty(B, H, T, dv, dtype=torch.float32, device=dev)
    _need(o, "o", (torch.float32,), (B, H, T, dv))
    D = D_out
    if D is None and want_D:
        D = torch.empty(B, H, T, dtype=torch.float32, device=dev)
    if D is not None:
        _need(D, "D", (torch.float32,), (B, H, T))
    S = z = None
    if want_state:
        S = torch.empty(B, H, F, dv, dtype=torch.float32, device=dev)
        z = torch.empty(B, H, F, dtype=torch.float32, device=dev)
    if S0 is not None:
        _need(S0, "S0", (torch.float32,), (B, H, F, dv))
        _need(z0, "z0", (torch.float32,), (B, H, F))
    ws_size = int(lib().sanatan_chunk_fwd_workspace_size(B, H, T, d, dv, _DT[q.dtype]))
    if workspace is None and ws_size > 0:
        workspace = torch.empty(ws_size, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().sanatan_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], _ptr(gamma),
                                 _ptr(omega), _ptr(phi), B, H, T, d, dv, int(pos0), float(eps),
                                 _ptr(S0), _ptr(z0), _ptr(o), _ptr(D), _ptr(S), _ptr(z),
                                 _ptr(workspace), ws_bytes, _stream(dev))
    _check("sanatan_chunk_fwd", st)
    return o, D, S, z


class HostForward:
    """sanatan_chunk_fwd over pinned HOST tensors q, k, v (bf16 [B, H, T, d])
    into a pinned host o (f32 [B, H, T, dv]), pipelined over slices of the B * H
    sequences: the host-to-device copy of slice i + 1, the attention of slice
    i and the device-to-host copy of slice i - 1 run on three CUDA streams at
    once (one cudaMemcpyAsync per tensor slice).  A slice is m = B * H / slices
    consecutive sequences: whole batch rows when H divides m, else m heads of
    one batch row (then m must divide H), with the matching rows of gamma,
    omega and phi.  Device staging (two slices of q, k, v and o, and the
    workspace) is allocated once, here, with torch; each call then allocates
    nothing.  The calling stream waits for the last copy, so `o` is complete
    once that stream is synchronised."""

    def __init__(self, B, H, T, d=64, dv=64, slices=4, device=None):
        n_seq = B * H
        if slices < 1 or n_seq % slices:
            raise ValueError("B * H must be a multiple of slices")
        m = n_seq // slices
        if not (m % H == 0 or H % m == 0):
            raise ValueError("a slice must hold whole batch rows or divide one")
        self.dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.B, self.H, self.T, self.d, self.dv, self.n, self.m = B, H, T, d, dv, slices, m
        # device shape of one slice
        self.shape = (m // H, H) if m % H == 0 else (1, m)
        sb, sh = self.shape
        mk = lambda dt, last: [torch.empty(sb, sh, T, last, dtype=dt, device=self.dev)  # noqa: E731
                               for _ in range(2)]
        self.q, self.k, self.v = mk(torch.bfloat16, d), mk(torch.bfloat16, d), mk(torch.bfloat16, dv)
        self.o = mk(torch.float32, dv)
        ws = chunk_fwd_workspace_size(sb, sh, T, d, dv)
        self.ws = torch.empty(max(ws, 16), dtype=torch.uint8, device=self.dev)
        self.s_in = torch.cuda.Stream(self.dev)
        self.s_run = torch.cuda.Stream(self.dev)
        self.s_out = torch.cuda.Stream(self.dev)
        self.loaded = [torch.cuda.Event() for _ in range(2)]
        self.done = [torch.cuda.Event() for _ in range(2)]
        self.freed_in = [torch.cuda.Event() for _ in range(2)]
        self.freed_out = [torch.cuda.Event() for _ in range(2)]
        # per head range of a sub-row slice: its own (16-byte aligned) copies of
        # gamma, omega, phi, refreshed at every call
        self.params = {}
        if sh < H:
            for h0 in range(0, H, sh):
                self.params[h0] = (torch.empty(sh, device=self.dev),
                                   torch.empty(sh, d, device=self.dev),
                                   torch.empty(sh, d, device=self.dev))

    def _part(self, t, i):
        """Slice i of a [B, H, ...] host tensor, shaped like the device slice."""
        sb, sh = self.shape
        if sh == self.H:
            return t[i * sb:(i + 1) * sb]
        b, h0 = divmod(i * sh, self.H)
        return t[b:b + 1, h0:h0 + sh]


    def __call__(self, qh, kh, vh, gamma, omega, phi, oh, pos0=0, eps=0.0):
        for t, n in ((qh, "q"), (kh, "k"), (vh, "v"), (oh, "o")):
            if t.is_cuda or not t.is_pinned():
                raise ValueError(f"{n} must be a pinned host tensor")
        caller = torch.cuda.current_stream(self.dev)
        for st in (self.s_in, self.s_run, self.s_out):
            st.wait_stream(caller)
        sh = self.shape[1]
        if self.params:
            with torch.cuda.stream(self.s_run):
                for h0, (g, w, f) in self.params.items():
                    g.copy_(gamma[h0:h0 + sh])
                    w.copy_(omega[h0:h0 + sh])
                    f.copy_(phi[h0:h0 + sh])
        for i in range(self.n + 2):
            j = i % 2
            if i < self.n:                      # H2D of slice i into buffer j
                with torch.cuda.stream(self.s_in):
                    if i >= 2:
                        self.s_in.wait_event(self.freed_in[j])
                    self.q[j].copy_(self._part(qh, i), non_blocking=True)
                    self.k[j].copy_(self._part(kh, i), non_blocking=True)
                    self.v[j].copy_(self._part(vh, i), non_blocking=True)
                    self.loaded[j].record(self.s_in)
            if 1 <= i <= self.n:                # attention of slice i - 1
                jj = (i - 1) % 2
                g, w, f = (gamma, omega, phi) if not self.params else \
                    self.params[((i - 1) * sh) % self.H]
                with torch.cuda.stream(self.s_run):
                    self.s_run.wait_event(self.loaded[jj])
                    if i - 1 >= 2:
                        self.s_run.wait_event(self.freed_out[jj])
                    sanatan_chunk_fwd(self.q[jj], self.k[jj], self.v[jj], g, w, f, pos0=pos0,
                                      eps=eps, want_D=False, out=self.o[jj], workspace=self.ws)
                    self.freed_in[jj].record(self.s_run)
                    self.done[jj].record(self.s_run)
            if i >= 2:                          # D2H of slice i - 2
                jj = (i - 2) % 2
                with torch.cuda.stream(self.s_out):
                    self.s_out.wait_event(self.done[jj])
                    self._part(oh, i - 2).copy_(self.o[jj], non_blocking=True)
                    self.freed_out[jj].record(self.s_out)
        caller.wait_stream(self.s_out)
        return oh

    def capture(self, qh, kh, vh, gamma, omega, phi, oh, pos0=0, eps=0.0):
        """Record one call on these (fixed) host and parameter tensors as a CUDA
        graph -- every copy and kernel of the pipeline, on its three streams --
        so that replay() enqueues the whole step with one launch.  The call is
        run once first (warm-up outside the capture)."""
        self(qh, kh, vh, gamma, omega, phi, oh, pos0, eps)
        torch.cuda.current_stream(self.dev).synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self(qh, kh, vh, gamma, omega, phi, oh, pos0, eps)
        return self

    def replay(self):
        """One step of the captured pipeline on the current stream."""
        self.graph.replay()


def sanatan_chunk_fwd_noalloc(q, k, v, gamma, omega, phi, pos0=0, eps=0.0, S0=None, z0=None,
                              want_D=True, want_state=False):
    """sanatan_chunk_fwd for bf16 inputs without a workspace: the library uses
    its own fixed 16 MiB device scratch instead (for callers that cannot
    allocate).  Calls must not overlap on the GPU.  Returns (o, D, S, z)."""
    _need(q, "q", (torch.bfloat16,))
    B, H, T, d = q.shape
    _need(k, "k", (torch.bfloat16,), (B, H, T, d))
    dv = v.shape[-1]
    _need(v, "v", (torch.bfloat16,), (B, H, T, dv))
    _need_params(gamma, omega, phi, H, d)
    dev = q.device
    F = 6 * d
    o = torch.empty(B, H, T, dv, dtype=torch.float32, device=dev)
    D = torch.empty(B, H, T, dtype=torch.float32, device=dev) if want_D else None
    S = z = None
    if want_state:
        S = torch.empty(B, H, F, dv, dtype=torch.float32, device=dev)
        z = torch.empty(B, H, F, dtype=torch.float32, device=dev)
    st = lib().sanatan_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(omega),
                                         _ptr(phi), B, H, T, d, dv, int(pos0), float(eps),
                                         _ptr(S0), _ptr(z0), _ptr(o), _ptr(D), _ptr(S), _ptr(z),
                                         _stream(dev))
    _check("sanatan_chunk_fwd_noalloc", st)
    return o, D, S, z


def power_fwd_workspace_size(B, H, T, d=64, dv=64):
    return int(lib().sanatan_power_fwd_workspace_size(B, H, T, d, dv))


def sanatan_power_fwd(q, k, v, gamma, omega, phi, p, pos0=0, eps=0.0, want_D=True, out=None,
                      D_out=None, workspace=None):
    """Power-sharpened causal attention at integer power p (bf16 q, k, v).

    Returns (o [B,H,T,dv] f32, D [B,H,T] f32 or None)."""
    _need(q, "q", (torch.bfloat16,))
    B, H, T, d = q.shape
    _need(k, "k", (torch.bfloat16,), (B, H, T, d))
    dv = v.shape[-1]
    _need(v, "v", (torch.bfloat16,), (B, H, T, dv))
    _need_params(gamma, omega, phi, H, d)
    dev = q.device
    o = out if out is not None else torch.empty(B, H, T, dv, dtype=torch.float32, device=dev)
    _need(o, "o", (torch.float32,), (B, H, T, dv))
    D = D_out
    if D is None and want_D:
        D = torch.empty(B, H, T, dtype=torch.float32, device=dev)
    if D is not None:
        _need(D, "D", (torch.float32,), (B, H, T))
    ws_size = power_fwd_workspace_size(B, H, T, d, dv)
    if workspace is None and ws_size > 0:
        workspace = torch.empty(ws_size, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().sanatan_power_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(omega), _ptr(phi),
                                 B, H, T, d, dv, int(pos0), int(p), float(eps), _ptr(o), _ptr(D),
                                 _ptr(workspace), ws_bytes, _stream(dev))
    _check("sanatan_power_fwd", st)
    return o, D


def power_bwd_workspace_size(B, H, T, d=64, dv=64):
    return int(lib().sanatan_power_bwd_workspace_size(B, H, T, d, dv))


def sanatan_power_bwd(q, k, v, gamma, omega, phi, p, o, D, dO, pos0=0, eps=0.0, want_dphi=True,
                      workspace=None):
    """Gradients of sum(o * dO) for sanatan_power_fwd (bf16 q, k, v).

    Returns a dict with dq, dk, dv (bf16), dgamma, domega and dphi (f32; dphi
    None unless want_dphi)."""
    _need(q, "q", (torch.bfloat16,))
    B, H, T, d = q.shape
    _need(k, "k", (torch.bfloat16,), (B, H, T, d))
    dv_ = v.shape[-1]
    _need(v, "v", (torch.bfloat16,), (B, H, T, dv_))
    _need(o, "o", (torch.float32,), (B, H, T, dv_))
    _need(D, "D", (torch.float32,), (B, H, T))
    _need(dO, "dO", (torch.float32, torch.bfloat16), (B, H, T, dv_))
    _need_params(gamma, omega, phi, H, d)
    dev = q.device
    dq, dk, dvo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dgamma = torch.empty(H, dtype=torch.float32, device=dev)
    domega = torch.empty(H, d, dtype=torch.float32, device=dev)
    dphi = torch.empty(H, d, dtype=torch.float32, device=dev) if want_dphi else None
    ws_size = power_bwd_workspace_size(B, H, T, d, dv_)
    if workspace is None and ws_size > 0:
        workspace = torch.empty(ws_size, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().sanatan_power_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(omega), _ptr(phi),
                                 B, H, T, d, dv_, int(pos0), int(p), float(eps), _ptr(o), _ptr(D),
                                 _ptr(dO), _DT[dO.dtype], _ptr(dq), _ptr(dk), _ptr(dvo),
                                 _ptr(dgamma), _ptr(domega), _ptr(dphi), _ptr(workspace),
                                 ws_bytes, _stream(dev))
    _check("sanatan_power_bwd", st)
    return dict(dq=dq, dk=dk, dv=dvo, dgamma=dgamma, domega=domega, dphi=dphi)


def sanatan_ablation_fwd(q, k, v, gamma, omega, phi, p, channels, shift=0.0, pos0=0, eps=0.0,
                         want_D=True, out=None, D_out=None, workspace=None):
    """Power-sharpened causal attention with the four-channel (clipped) or the
    three-channel (optionally shifted) ablation map; bf16 q, k, v, p in {1, 2, 4}.

    Returns (o [B,H,T,dv] f32, D [B,H,T] f32 or None)."""
    _need(q, "q", (torch.bfloat16,))
    B, H, T, d = q.shape
    _need(k, "k", (torch.bfloat16,), (B, H, T, d))
    dv = v.shape[-1]
    _need(v, "v", (torch.bfloat16,), (B, H, T, dv))
    _need_params(gamma, omega, phi, H, d)
    dev = q.device
    o = out if out is not None else torch.empty(B, H, T, dv, dtype=torch.float32, device=dev)
    _need(o, "o", (torch.float32,), (B, H, T, dv))
    D = D_out
    if D is None and want_D:
        D = torch.empty(B, H, T, dtype=torch.float32, device=dev)
    if D is not None:
        _need(D, "D", (torch.float32,), (B, H, T))
    ws_size = power_fwd_workspace_size(B, H, T, d, dv)
    if workspace is None and ws_size > 0:
        workspace = torch.empty(ws_size, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().sanatan_ablation_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(omega),
                                    _ptr(phi), B, H, T, d, dv, int(pos0), int(p), int(channels),
                                    float(shift), float(eps), _ptr(o), _ptr(D), _ptr(workspace),
                                    ws_bytes, _stream(dev))
    _check("sanatan_ablation_fwd", st)
    return o, D


def chunk_bwd_workspace_size(B, H, T, d=64, dv=64, dtype=torch.bfloat16):
    return int(lib().sanatan_chunk_bwd_workspace_size(B, H, T, d, dv, _DT[dtype]))


def sanatan_chunk_bwd(q, k, v, gamma, omega, phi, o, D, dO, pos0=0, eps=0.0, S0=None, z0=None,
                      want_dphi=False, workspace=None, fwd_workspace=None):
    """Gradients of sum(o * dO): dict(dq, dk, dv, dgamma, domega, dphi).

    fwd_workspace: the workspace the forward that produced o and D ran with (on
    these same inputs), so that its per-segment state sums are reused."""
    _need(q, "q", (torch.float32, torch.bfloat16))
    B, H, T, d = q.shape
    dv = v.shape[-1]
    _need(k, "k", (q.dtype,), (B, H, T, d))
    _need(v, "v", (q.dtype,), (B, H, T, dv))
    _need(o, "o", (torch.float32,), (B, H, T, dv))
    _need(D, "D", (torch.float32,), (B, H, T))
    _need(dO, "dO", (torch.float32, torch.bfloat16), (B, H, T, dv))
    _need_params(gamma, omega, phi, H, d)
    dev = q.device
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dvv = torch.empty_like(v)
    dgamma = torch.empty(H, dtype=torch.float32, device=dev)
    domega = torch.empty(H, d, dtype=torch.float32, device=dev)
    dphi = torch.empty(H, d, dtype=torch.float32, device=dev) if want_dphi else None
    ws_size = int(lib().sanatan_chunk_bwd_workspace_size(B, H, T, d, dv, _DT[q.dtype]))
    if workspace is None and ws_size > 0:
        workspace = torch.empty(ws_size, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().sanatan_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], _ptr(gamma),
                                 _ptr(omega), _ptr(phi), B, H, T, d, dv, int(pos0), float(eps),
                                 _ptr(S0), _ptr(z0), _ptr(o), _ptr(D), _ptr(dO), _DT[dO.dtype],
                                 _ptr(dq), _ptr(dk), _ptr(dvv), _ptr(dgamma), _ptr(domega),
                                 _ptr(dphi), _ptr(workspace), ws_bytes, _ptr(fwd_workspace),
                                 0 if fwd_workspace is None else
                                 fwd_workspace.numel() * fwd_workspace.element_size(),
                                 _stream(dev))
    _check("sanatan_chunk_bwd", st)
    return dict(dq=dq, dk=dk, dv=dvv, dgamma=dgamma, domega=domega, dphi=dphi)


def sanatan_decode_step(S, z, q, k, v, gamma, omega, phi, pos, eps=0.0, out=None):
    """One decode token for N slots; S [N,6d,dv] and z [N,6d] are updated in
    place.  Returns o [N, dv] f32."""
    _need(q, "q", (torch.float32,))
    N, d = q.shape
    _need(k, "k", (torch.float32,), (N, d))
    _need(v, "v", (torch.float32,))
    dv = v.shape[-1]
    F = 6 * d
    _need(S, "S", (torch.float32,), (N, F, dv))
    _need(z, "z", (torch.float32,), (N, F))
    _need(pos, "pos", (torch.int64,), (N,))
    G = gamma.shape[0]
    _need(gamma, "gamma", (torch.float32,), (G,))
    _need(omega, "omega", (torch.float32,), (G, d))
    _need(phi, "phi", (torch.float32,), (G, d))
    o = out if out is not None else torch.empty(N, dv, dtype=torch.float32, device=q.device)
    _need(o, "o", (torch.float32,), (N, dv))
    st = lib().sanatan_decode_step(_ptr(S), _ptr(z), _ptr(q), _ptr(k), _ptr(v), _ptr(gamma),
                                   _ptr(omega), _ptr(phi), _ptr(pos), N, G, d, dv, float(eps),
                                   _ptr(o), _stream(q.device))
    _check("sanatan_decode_step", st)
    return o


def sanatan_stack_decode_step(x, Wqkv, Wo, S, z, gamma, omega, phi, pos, eps=0.0,
                              workspace=None):
    """One token through L attention layers; x [B, heads*64] is updated in
    place (and returned), S [L, B*heads, 384, 64] and z [L, B*heads, 384] too.
    gamma [L, heads], omega and phi [L, heads, 64], pos [B*heads] int64."""
    _need(x, "x", (torch.float32,))
    B, Dm = x.shape
    L, heads = gamma.shape
    d = Dm // heads
    _need(Wqkv, "Wqkv", (torch.float32,), (L, Dm, 3 * Dm))
    _need(Wo, "Wo", (torch.float32,), (L, Dm, Dm))
    _need(S, "S", (torch.float32,), (L, B * heads, 6 * d, d))
    _need(z, "z", (torch.float32,), (L, B * heads, 6 * d))
    _need(gamma, "gamma", (torch.float32,), (L, heads))
    _need(omega, "omega", (torch.float32,), (L, heads, d))
    _need(phi, "phi", (torch.float32,), (L, heads, d))
    _need(pos, "pos", (torch.int64,), (B * heads,))
    ws_n = int(lib().sanatan_stack_decode_workspace_size(B, heads, d))
    if workspace is None:
        workspace = torch.empty(max(ws_n, 16), dtype=torch.uint8, device=x.device)
    _check("sanatan_stack_decode_step",
           lib().sanatan_stack_decode_step(_ptr(x), _ptr(Wqkv), _ptr(Wo), _ptr(S), _ptr(z),
                                           _ptr(gamma), _ptr(omega), _ptr(phi), _ptr(pos), B, L,
                                           heads, d, float(eps), _ptr(workspace),
                                           workspace.numel(), _stream(x.device)))
    return x


def harmonic_features(harmonics, d=64):
    """F_N = 2 (2N + 1) d features of the harmonic map."""
    return 2 * (2 * harmonics + 1) * d


def sanatan_featurize_harmonic(u, gamma, omega, phi, harmonics, pos0=0, out_dtype=None):
    """Phi_N(u) [B, H, T, F_N] of the harmonic map."""
    _need(u, "u", (torch.float32, torch.bfloat16))
    B, H, T, d = u.shape
    _need_params(gamma, omega, phi, H, d)
    out = torch.empty(B, H, T, harmonic_features(harmonics, d), dtype=out_dtype or torch.float32,
                      device=u.device)
    _check("sanatan_featurize_harmonic",
           lib().sanatan_featurize_harmonic(_ptr(u), _DT[u.dtype], _ptr(gamma), _ptr(omega),
                                            _ptr(phi), B, H, T, d, int(pos0), int(harmonics),
                                            _ptr(out), _DT[out.dtype], _stream(u.device)))
    return out


def sanatan_chunk_fwd_harmonic(q, k, v, gamma, omega, phi, harmonics, pos0=0, eps=0.0, S0=None,
                               z0=None, want_D=True, want_state=False):
    """Causal p=1 attention with the harmonic map (float32 on the CUDA cores).
    Returns (o, D or None, S [B,H,F_N,dv] or None, z [B,H,F_N] or None)."""
    _need(q, "q", (torch.float32, torch.bfloat16))
    B, H, T, d = q.shape
    _need(k, "k", (q.dtype,), (B, H, T, d))
    dv = v.shape[-1]
    _need(v, "v", (q.dtype,), (B, H, T, dv))
    _need_params(gamma, omega, phi, H, d)
    F = harmonic_features(harmonics, d)
    dev = q.device
    o = torch.empty(B, H, T, dv, dtype=torch.float32, device=dev)
    D = torch.empty(B, H, T, dtype=torch.float32, device=dev) if want_D else None
    Sx = zx = None
    if want_state:
        Sx = torch.empty(B, H, F, dv, dtype=torch.float32, device=dev)
        zx = torch.empty(B, H, F, dtype=torch.float32, device=dev)
    if S0 is not None:
        _need(S0, "S0", (torch.float32,), (B, H, F, dv))
        _need(z0, "z0", (torch.float32,), (B, H, F))
    _check("sanatan_chunk_fwd_harmonic",
           lib().sanatan_chunk_fwd_harmonic(_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], _ptr(gamma),
                                            _ptr(omega), _ptr(phi), B, H, T, d, dv, int(pos0),
                                            int(harmonics), float(eps), _ptr(S0), _ptr(z0),
                                            _ptr(o), _ptr(D), _ptr(Sx), _ptr(zx), _stream(dev)))
    return o, D, Sx, zx


def sanatan_chunk_bwd_harmonic(q, k, v, gamma, omega, phi, harmonics, o, D, dO, pos0=0, eps=0.0,
                               S0=None, z0=None, want_dphi=False, workspace=None):
    """Gradients of sum(o * dO) for sanatan_chunk_fwd_harmonic: dict(dq, dk, dv,
    dgamma, domega, dphi)."""
    _need(q, "q", (torch.float32, torch.bfloat16))
    B, H, T, d = q.shape
    dv = v.shape[-1]
    _need(k, "k", (q.dtype,), (B, H, T, d))
    _need(v, "v", (q.dtype,), (B, H, T, dv))
    _need(o, "o", (torch.float32,), (B, H, T, dv))
    _need(D, "D", (torch.float32,), (B, H, T))
    _need(dO, "dO", (torch.float32, torch.bfloat16), (B, H, T, dv))
    _need_params(gamma, omega, phi, H, d)
    dev = q.device
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dvv = torch.empty_like(v)
    dgamma = torch.empty(H, dtype=torch.float32, device=dev)
    domega = torch.empty(H, d, dtype=torch.float32, device=dev)
    dphi = torch.empty(H, d, dtype=torch.float32, device=dev) if want_dphi else None
    ws_size = int(lib().sanatan_chunk_bwd_harmonic_workspace_size(B, H, T, d, dv,
                                                                   int(harmonics)))
    if workspace is None and ws_size > 0:
        workspace = torch.empty(ws_size, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().sanatan_chunk_bwd_harmonic(_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], _ptr(gamma),
                                          _ptr(omega), _ptr(phi), B, H, T, d, dv, int(pos0),
                                          int(harmonics), float(eps), _ptr(S0), _ptr(z0), _ptr(o),
                                          _ptr(D), _ptr(dO), _DT[dO.dtype], _ptr(dq), _ptr(dk),
                                          _ptr(dvv), _ptr(dgamma), _ptr(domega), _ptr(dphi),
                                          _ptr(workspace), ws_bytes, _stream(dev))
    _check("sanatan_chunk_bwd_harmonic", st)
    return dict(dq=dq, dk=dk, dv=dvv, dgamma=dgamma, domega=domega, dphi=dphi)


def sanatan_decode_step_harmonic(S, z, q, k, v, gamma, omega, phi, pos, harmonics, eps=0.0):
    """One decode token with the harmonic map; S [N,F_N,dv], z [N,F_N] in place."""
    _need(q, "q", (torch.float32,))
    N, d = q.shape
    _need(k, "k", (torch.float32,), (N, d))
    dv = v.shape[-1]
    _need(v, "v", (torch.float32,), (N, dv))
    F = harmonic_features(harmonics, d)
    _need(S, "S", (torch.float32,), (N, F, dv))
    _need(z, "z", (torch.float32,), (N, F))
    _need(pos, "pos", (torch.int64,), (N,))
    G = gamma.shape[0]
    _need_params(gamma, omega, phi, G, d)
    o = torch.empty(N, dv, dtype=torch.float32, device=q.device)
    _check("sanatan_decode_step_harmonic",
           lib().sanatan_decode_step_harmonic(_ptr(S), _ptr(z), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(gamma), _ptr(omega), _ptr(phi), _ptr(pos), N,
                                              G, d, dv, int(harmonics), float(eps), _ptr(o),
                                              _stream(q.device)))
    return o


SCAN_GATES = {"log": 0, "sigmoid": 1}
SCAN_MARK = 64    # tokens between two saved states of the gated recurrence
CACHE_GROUP = 64  # values that share a scale in the state cache
_CACHE_FMT = {torch.int8: 0, torch.float8_e4m3fn: 1}


def _gate(gate):
    if gate not in SCAN_GATES:
        raise ValueError(f"gate must be one of {tuple(SCAN_GATES)}, not {gate!r}")
    return SCAN_GATES[gate]


def _fit(t, name, dtype, shape, dev):
    """t on the device, contiguous, of this type and shape (_need's checks, the
    usual answer first: small calls are bound by the host)."""
    if t.__class__ is torch.Tensor and t.dtype is dtype and t.shape == shape and \
            t.device == dev and t.is_contiguous():
        return t
    _need(t, name, (dtype,), shape)
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return t


def _at(t):
    return None if t is None else t.data_ptr()


def _at16(t):
    """t, or a copy of it where it does not start at 16 bytes: a part of a longer
    list, one sequence's state of a batch's, a gradient cut out of a larger one."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.detach().clone()


def _call(name, dev, *args):
    """Call a library function with the tensors' device current, on its stream
    (asked for raw: a Stream object costs as much as the launch)."""
    fn = getattr(lib(), name)
    if dev.index == torch.cuda.current_device():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        raise SanatanError(name, st)


def _scan_args(x, g, gate, lens, dims):
    """x, g and lens fit; returns (x's shape, device, dtype code, gate code)."""
    _need(x, "x", _FLOATS)
    if x.dim() != dims:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected {dims} dimensions")
    shape, dev = x.shape, x.device
    _fit(g, "g", x.dtype, shape, dev)
    if lens is not None:
        _fit(lens, "lens", torch.int64, (shape[0],), dev)
    return shape, dev, _DT[x.dtype], _gate(gate)


def sanatan_gated_scan_fwd(x, g, gate="log", h0=None, lens=None, want_state=False,
                           want_marks=False, out=None, h_out=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t over x, g [B, T, D] (f32
    or bf16): gate "log" has a = exp(g), u = x, gate "sigmoid" a = 1 / (1 +
    exp(-g)), u = (1 - a) x.  h0 [B, D] f32 is the state before the first
    token; tokens from lens[b] (int64 [B]) on are left out and give zeros.
    lens, h0 and h_out may be parts of larger tensors (copied where the library
    needs them at 16 bytes).

    Returns (y [B,T,D] in x's dtype, the last state [B,D] f32 or None, marks
    [B, ceil(T/64), D] f32 (states for the backward) or None)."""
    (B, T, D), dev, dt, gt = _scan_args(x, g, gate, lens, 3)
    y = torch.empty_like(x) if out is None else _fit(out, "out", x.dtype, x.shape, dev)
    if h0 is not None:
        _fit(h0, "h0", torch.float32, (B, D), dev)
    if h_out is not None:
        _fit(h_out, "h_out", torch.float32, (B, D), dev)
    elif want_state:
        h_out = torch.empty(B, D, dtype=torch.float32, device=dev)
    marks = torch.empty(B, -(-T // SCAN_MARK), D, dtype=torch.float32, device=dev) \
        if want_marks else None
    lens, h0 = _at16(lens), _at16(h0)
    last = _at16(h_out)
    _call("sanatan_gated_scan_fwd", dev, x.data_ptr(), g.data_ptr(), dt, gt, _at(lens), B, T, D,
          _at(h0), y.data_ptr(), _at(last), _at(marks))
    if last is not h_out:
        h_out.detach().copy_(last)
    return y, h_out, marks


def sanatan_gated_scan_bwd(x, g, dy, marks, gate="log", lens=None, dh_last=None, want_dh0=False):
    """Gradients of sum(y * dy) + sum(h_last * dh_last) for
    sanatan_gated_scan_fwd: dict(dx, dg, dh0); marks are the forward's."""
    (B, T, D), dev, dt, gt = _scan_args(x, g, gate, lens, 3)
    _fit(dy, "dy", x.dtype, x.shape, dev)
    _fit(marks, "marks", torch.float32, (B, -(-T // SCAN_MARK), D), dev)
    if dh_last is not None:
        _fit(dh_last, "dh_last", torch.float32, (B, D), dev)
    dx, dg = torch.empty_like(x), torch.empty_like(g)
    dh0 = torch.empty(B, D, dtype=torch.float32, device=dev) if want_dh0 else None
    lens, dh_last = _at16(lens), _at16(dh_last)
    _call("sanatan_gated_scan_bwd", dev, x.data_ptr(), g.data_ptr(), dy.data_ptr(), dt, gt,
          _at(lens), B, T, D, marks.data_ptr(), _at(dh_last), dx.data_ptr(), dg.data_ptr(),
          _at(dh0))
    return dict(dx=dx, dg=dg, dh0=dh0)


def sanatan_gated_scan_step(h, x, g, gate="log", out=None):
    """One token of the gated recurrence for N sequences: h [N, D] f32 is
    updated in place, x and g [N, D] f32 or bf16.  Returns y [N, D]."""
    (N, D), dev, dt, gt = _scan_args(x, g, gate, None, 2)
    _fit(h, "h", torch.float32, x.shape, dev)
    y = torch.empty_like(x) if out is None else _fit(out, "out", x.dtype, x.shape, dev)
    _call("sanatan_gated_scan_step", dev, h.data_ptr(), x.data_ptr(), g.data_ptr(), dt, gt, N, D,
          y.data_ptr())
    return y


class GatedScan(torch.autograd.Function):
    """autograd wrapper: (y, h_last) = GatedScan.apply(x, g, gate, h0, lens);
    forward = sanatan_gated_scan_fwd, backward = sanatan_gated_scan_bwd."""

    @staticmethod
    def forward(ctx, x, g, gate="log", h0=None, lens=None):
        y, h, marks = sanatan_gated_scan_fwd(x, g, gate, h0=h0, lens=lens, want_state=True,
                                             want_marks=any(ctx.needs_input_grad))
        ctx.save_for_backward(x, g, marks, lens)
        ctx.gate = gate
        ctx.want_dh0 = h0 is not None and ctx.needs_input_grad[3]
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_last):
        x, g, marks, lens = ctx.saved_tensors
        if dy is None and dh_last is None:
            return None, None, None, None, None
        dy = torch.zeros_like(x) if dy is None else dy.contiguous()
        dh_last = None if dh_last is None else dh_last.contiguous()
        d = sanatan_gated_scan_bwd(x, g, dy, marks, ctx.gate, lens=lens, dh_last=dh_last,
                                   want_dh0=ctx.want_dh0)
        return d["dx"], d["dg"], None, d["dh0"], None


def _stretch(t, name, layers, B):
    """Values of one sequence's layer in t, read as [layers, B, ...]."""
    n, total = layers * B, t.numel()
    if n == 0 and total == 0:
        return 0
    if n == 0 or total % n:
        raise ValueError(f"{name} has shape {tuple(t.shape)}: not {layers} layers of {B} "
                         "sequences")
    return total // n


def _cache_args(state, pages, codes, scales, z, z_cache, layers, name):
    """Checks shared by the two directions; returns (B, inner, z's inner, P, format)."""
    _need(state, name, (torch.float32,))
    dev = state.device
    if layers < 1 or pages.dim() != 1 or codes.dim() != 4 or codes.dtype not in _CACHE_FMT:
        raise ValueError("layers must be 1 or more, pages [B] and codes [P, layers, groups, 64] "
                         f"of a type in {tuple(_CACHE_FMT)}")
    B, P = pages.shape[0], codes.shape[0]
    _fit(pages, "pages", torch.int64, (B,), dev)
    inner, zi = _stretch(state, name, layers, B), 0
    if B:
        groups = -(-inner // CACHE_GROUP)
        _fit(codes, "codes", codes.dtype, (P, layers, groups, CACHE_GROUP), dev)
        _fit(scales, "scales", torch.float32, (P, layers, groups), dev)
    if (z is None) != (z_cache is None):
        raise ValueError("z and z_cache go together")
    if z is not None:
        _fit(z, "z", torch.float32, z.shape, dev)
        zi = _stretch(z, "z", layers, B)
        if B:
            _fit(z_cache, "z_cache", torch.float32, (P, layers, zi), dev)
    return B, inner, zi, P, _CACHE_FMT[codes.dtype]


def state_cache_empty(pages, inner, z_inner=0, layers=1, dtype=torch.int8, device=None):
    """A pool of zeroed pages: (codes [pages, layers, ceil(inner/64), 64] int8 or
    float8_e4m3fn, scales f32, z_cache [pages, layers, z_inner] f32 or None)."""
    if dtype not in _CACHE_FMT:
        raise ValueError(f"dtype must be one of {tuple(_CACHE_FMT)}, not {dtype}")
    groups = -(-int(inner) // CACHE_GROUP)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    codes = torch.zeros(pages, layers, groups, CACHE_GROUP, dtype=torch.int8, device=dev)
    scales = torch.zeros(pages, layers, groups, dtype=torch.float32, device=dev)
    zc = torch.zeros(pages, layers, z_inner, dtype=torch.float32, device=dev) if z_inner else None
    return codes.view(dtype), scales, zc


def sanatan_state_cache_write(state, pages, codes, scales, z=None, z_cache=None, layers=1):
    """Keep the float32 states of B sequences in the pages[b] of a pool (int8 or
    e4m3 codes with a scale per 64 values; z in float32).  state is read as
    [layers, B, inner] and z as [layers, B, z_inner] (any shape of that many
    values, e.g. the S and z of sanatan_chunk_fwd, of decode slots in
    sequence-major order, or, with layers = L, of the stack decode); pages [B]
    int64, where a value outside the pool leaves the sequence out.  See
    include/sanatan.h for the formats."""
    B, inner, zi, P, fmt = _cache_args(state, pages, codes, scales, z, z_cache, layers, "state")
    _call("sanatan_state_cache_write", state.device, state.data_ptr(), _at(z), layers, B, inner,
          zi, pages.data_ptr(), P, fmt, codes.data_ptr(), scales.data_ptr(), _at(z_cache))


def sanatan_state_cache_read(codes, scales, pages, state, z_cache=None, z=None, layers=1):
    """Take the states of B sequences up from the pages[b] of a pool into state
    (and z), laid out as for sanatan_state_cache_write.  A page may serve
    several sequences; sequences whose page is outside the pool keep what state
    holds.  Returns state."""
    B, inner, zi, P, fmt = _cache_args(state, pages, codes, scales, z, z_cache, layers, "state")
    _call("sanatan_state_cache_read", state.device, codes.data_ptr(), scales.data_ptr(),
          _at(z_cache), P, fmt, pages.data_ptr(), layers, B, inner, zi, state.data_ptr(), _at(z))
    return state


class SanatanAttention(torch.autograd.Function):
    """autograd wrapper: forward = sanatan_chunk_fwd, backward = sanatan_chunk_bwd."""

    @staticmethod
    def forward(ctx, q, k, v, gamma, omega, phi, pos0=0, eps=0.0):
        B, H, T, d = q.shape
        ws_size = chunk_fwd_workspace_size(B, H, T, d, v.shape[-1], q.dtype)
        ws = torch.empty(max(ws_size, 16), dtype=torch.uint8, device=q.device)
        o, D, _, _ = sanatan_chunk_fwd(q, k, v, gamma, omega, phi, pos0=pos0, eps=eps,
                                       workspace=ws)
        ctx.save_for_backward(q, k, v, gamma, omega, phi, o, D)
        ctx.pos0, ctx.eps = pos0, eps
        ctx.fwd_ws = ws   # its per-segment state sums serve the backward
        return o

    @staticmethod
    def backward(ctx, dO):
        q, k, v, gamma, omega, phi, o, D = ctx.saved_tensors
        g = sanatan_chunk_bwd(q, k, v, gamma, omega, phi, o, D, dO.contiguous(), pos0=ctx.pos0,
                              eps=ctx.eps, want_dphi=True, fwd_workspace=ctx.fwd_ws)
        return g["dq"], g["dk"], g["dv"], g["dgamma"], g["domega"], g["dphi"], None, None
