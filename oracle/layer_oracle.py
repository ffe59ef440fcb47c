"""Float64 definitions of the layer norm, the short causal convolution and the
selective scan.

Plain NumPy, one sequence and one token at a time; test infrastructure only, it
shares no code with the library.

Layer norm (rows s of D values): y = (s - mean) / sqrt(var + eps) w + b.
Short causal convolution: c_t = bias + sum_k w_k x_{t-K+1+k}, where x before the
first token is the state; y = c, or c / (1 + exp(-c)).
Selective scan: delta = dt + dt_bias or log(1 + exp(dt + dt_bias)),
    h_t = exp(delta A) h_{t-1} + delta u B_t,
    y_t = (sum_n C_t h_t + D u) z / (1 + exp(-z)).
"""
import numpy as np


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def silu_slope(x):
    s = sigmoid(x)
    return s * (1 + x * (1 - s))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def lengths(lens, B, T):
    return [T] * B if lens is None else [min(max(int(n), 0), T) for n in lens]


def layer_norm(s, w=None, b=None, eps=1e-5):
    """s [rows, D] -> (y, mean [rows], 1 / sqrt(var + eps) [rows])."""
    mean = s.mean(-1)
    rstd = 1 / np.sqrt(((s - mean[:, None]) ** 2).mean(-1) + eps)
    hat = (s - mean[:, None]) * rstd[:, None]
    return hat * (1 if w is None else w) + (0 if b is None else b), mean, rstd


def layer_norm_backward(s, w, dy, ds=None, eps=1e-5):
    """Gradients (dx, dw, db) of sum(y dy) + sum(s ds)."""
    _, mean, rstd = layer_norm(s, eps=eps)
    hat = (s - mean[:, None]) * rstd[:, None]
    g = dy * (1 if w is None else w)
    dx = rstd[:, None] * (g - g.mean(-1, keepdims=True) - hat * (g * hat).mean(-1, keepdims=True))
    return dx + (0 if ds is None else ds), (dy * hat).sum(0), dy.sum(0)


def causal_conv(x, w, bias=None, silu=True, s0=None, lens=None):
    """x [B, T, D], w [D, K] -> (y, last inputs [B, K - 1, D], c)."""
    B, T, D = x.shape
    K = w.shape[1]
    y, c, last = np.zeros((B, T, D)), np.zeros((B, T, D)), np.zeros((B, K - 1, D))
    for b, n in enumerate(lengths(lens, B, T)):
        row = np.concatenate([np.zeros((K - 1, D)) if s0 is None else s0[b], x[b, :n]])
        for t in range(n):
            c[b, t] = (0 if bias is None else bias) + (w.T * row[t:t + K]).sum(0)
            y[b, t] = c[b, t] * sigmoid(c[b, t]) if silu else c[b, t]
        last[b] = row[n:]
    return y, last, c


def causal_conv_backward(x, w, dy, bias=None, silu=True, s0=None, lens=None, ds_last=None):
    """Gradients (dx, dw, dbias, ds0) of sum(y dy) + sum(last ds_last)."""
    B, T, D = x.shape
    K = w.shape[1]
    _, _, c = causal_conv(x, w, bias, silu, s0, lens)
    dx, dw, db, ds0 = np.zeros((B, T, D)), np.zeros((D, K)), np.zeros(D), np.zeros((B, K - 1, D))
    for b, n in enumerate(lengths(lens, B, T)):
        row = np.concatenate([np.zeros((K - 1, D)) if s0 is None else s0[b], x[b, :n]])
        d = np.zeros_like(row)
        for t in range(n):
            dc = dy[b, t] * (silu_slope(c[b, t]) if silu else 1)
            d[t:t + K] += w.T * dc
            dw += (row[t:t + K] * dc).T
            db += dc
        if ds_last is not None:
            d[n:] += ds_last[b]
        dx[b, :n], ds0[b] = d[K - 1:], d[:K - 1]
    return dx, dw, db, ds0


def selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, soft=True, h0=None, lens=None):
    """u, dt [b, T, width], A [width, N], B, C [b, T, N] -> (y, h_last, states before every
    token [b, T, width, N])."""
    b, T, width = u.shape
    N = A.shape[1]
    y, before = np.zeros((b, T, width)), np.zeros((b, T, width, N))
    h = np.zeros((b, width, N)) if h0 is None else np.array(h0, dtype=np.float64)
    for i, n in enumerate(lengths(lens, b, T)):
        for t in range(T):
            before[i, t] = h[i]
            if t >= n:
                continue
            raw = dt[i, t] + (0 if dt_bias is None else dt_bias)
            delta = softplus(raw) if soft else raw
            h[i] = np.exp(delta[:, None] * A) * h[i] + (delta * u[i, t])[:, None] * B[i, t]
            y[i, t] = h[i] @ C[i, t] + (0 if D is None else D * u[i, t])
            if z is not None:
                y[i, t] *= z[i, t] * sigmoid(z[i, t])
    return y, h, before


def selective_scan_backward(u, dt, A, B, C, dy, D=None, z=None, dt_bias=None, soft=True, h0=None,
                            lens=None, dh_last=None):
    """Gradients of sum(y dy) + sum(h_last dh_last): dict."""
    b, T, width = u.shape
    _, _, before = selective_scan(u, dt, A, B, C, D, z, dt_bias, soft, h0, lens)
    out = {k: np.zeros((b, T, width)) for k in ("du", "ddt", "dz")}
    out.update(dA=np.zeros(A.shape), dB=np.zeros(B.shape), dC=np.zeros(C.shape),
               dD=np.zeros(width), ddt_bias=np.zeros(width))
    g = np.zeros((b, *A.shape)) if dh_last is None else np.array(dh_last, dtype=np.float64)
    for i, n in enumerate(lengths(lens, b, T)):
        for t in range(n - 1, -1, -1):
            raw = dt[i, t] + (0 if dt_bias is None else dt_bias)
            delta = softplus(raw) if soft else raw
            a = np.exp(delta[:, None] * A)
            h = a * before[i, t] + (delta * u[i, t])[:, None] * B[i, t]
            v = dy[i, t]
            if z is not None:
                y0 = h @ C[i, t] + (0 if D is None else D * u[i, t])
                out["dz"][i, t] = v * y0 * silu_slope(z[i, t])
                v = v * z[i, t] * sigmoid(z[i, t])
            dh = g[i] + v[:, None] * C[i, t]
            out["dC"][i, t] = v @ h
            out["dB"][i, t] = (delta * u[i, t]) @ dh
            g[i] = a * dh
            w = g[i] * before[i, t]
            out["dA"] += delta[:, None] * w
            out["du"][i, t] = delta * (dh @ B[i, t]) + (0 if D is None else D * v)
            ddelta = u[i, t] * (dh @ B[i, t]) + (w * A).sum(-1)
            out["ddt"][i, t] = ddelta * (sigmoid(raw) if soft else 1)
            out["dD"] += v * u[i, t]
            out["ddt_bias"] += out["ddt"][i, t]
    out["dh0"] = g
    return out
