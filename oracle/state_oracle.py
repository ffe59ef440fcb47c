"""Float64 definitions of the gated linear recurrence and of the state cache.

Plain NumPy, one token and one group at a time; test infrastructure only, it
shares no code with the library.

Gated recurrence (per channel; a the decay, u the input):
    h_t = a_t h_{t-1} + u_t,  y_t = h_t
    "log":      a = exp(g),              u = x
    "sigmoid":  a = 1 / (1 + exp(-g)),   u = (1 - a) x
State cache (per group of 64 values x): "int8" s = max|x| / 127 in float32 and
the integer nearest x / s; "e4m3" s the smallest power of two with max|x| / s
<= 448 and x / s in e4m3.  Ties go to the even code.
"""
import numpy as np

GROUP = 64
TINY = 2.0 ** -100    # smaller groups are stored as zeros
LARGE = 2.0 ** 127    # larger ones as NaN


def gates(x, g, gate):
    """(a, 1 - a, u) of the two gates (the log gate's input has no factor)."""
    if gate == "log":
        return np.exp(g), np.ones_like(g), x
    with np.errstate(over="ignore"):
        a, keep = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    return a, keep, keep * x


def _present(lens, B, T):
    if lens is None:
        return np.ones((B, T), bool)
    return np.arange(T)[None] < np.asarray(lens)[:, None]


def gated_scan(x, g, gate, h0=None, lens=None):
    """x, g [B, T, D] -> (y [B, T, D], h_last [B, D], h_before [B, T, D])."""
    B, T, D = x.shape
    a, _, u = gates(x, g, gate)
    there = _present(lens, B, T)
    h = np.zeros((B, D)) if h0 is None else np.array(h0, dtype=np.float64)
    y, before = np.zeros((B, T, D)), np.zeros((B, T, D))
    for t in range(T):
        before[:, t] = h
        m = there[:, t][:, None]
        with np.errstate(invalid="ignore"):
            h = np.where(m, a[:, t] * h + u[:, t], h)
        y[:, t] = np.where(m, h, 0.0)
    return y, h, before


def gated_scan_backward(x, g, gate, dy, h0=None, lens=None, dh_last=None):
    """Gradients (dx, dg, dh0) of sum(y dy) + sum(h_last dh_last)."""
    B, T, D = x.shape
    a, keep, _ = gates(x, g, gate)
    _, _, before = gated_scan(x, g, gate, h0, lens)
    there = _present(lens, B, T)
    dh = np.zeros((B, D)) if dh_last is None else np.array(dh_last, dtype=np.float64)
    dx, dg = np.zeros((B, T, D)), np.zeros((B, T, D))
    for t in range(T - 1, -1, -1):
        m = there[:, t][:, None]
        d = dh + dy[:, t]
        if gate == "log":
            gx, gg = d, d * a[:, t] * before[:, t]
        else:
            gx = d * keep[:, t]
            gg = d * (before[:, t] - x[:, t]) * a[:, t] * keep[:, t]
        dx[:, t], dg[:, t] = np.where(m, gx, 0.0), np.where(m, gg, 0.0)
        dh = np.where(m, a[:, t] * d, dh)
    return dx, dg, dh


def gated_scan_step(h, x, g, gate):
    """One token: the new state [N, D], which is also the output."""
    a, _, u = gates(x, g, gate)
    return a * h + u


def e4m3_round(v):
    """v to the nearest e4m3 value (4 exponent bits, bias 7, 3 mantissa bits, no
    infinity, largest 448), ties to the even mantissa; |v| <= 464."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    return np.rint(v / step) * step


def cache_groups(x):
    """[..., inner] -> [..., groups, 64], filled up with zeros."""
    x = np.asarray(x, dtype=np.float64)
    fill = -x.shape[-1] % GROUP
    x = np.concatenate([x, np.zeros(x.shape[:-1] + (fill,))], -1)
    return x.reshape(x.shape[:-1] + (-1, GROUP))


def cache_store(x, fmt):
    """(codes as values, scales) of [..., inner] float32 values."""
    x = cache_groups(x)
    with np.errstate(invalid="ignore"):
        top = np.abs(x).max(-1)
    bad = ~(np.abs(x) < LARGE).all(-1)
    top = np.where(bad, 0.0, top)
    if fmt == "int8":
        s = np.float32(top / 127).astype(np.float64)
    else:
        m, e = np.frexp(top)
        s = np.ldexp(1.0, np.where(m > 0.875, e - 8, e - 9))
    s = np.where(top < TINY, 0.0, s)
    one = np.where(s == 0, 1.0, s)[..., None]
    with np.errstate(invalid="ignore"):
        q = np.where((s == 0)[..., None], 0.0, x / one)
    c = np.rint(q) if fmt == "int8" else e4m3_round(q)
    return np.where(bad[..., None], 0.0, c), np.where(bad, np.nan, s)


def cache_values(codes, scales, inner):
    """What a reader gets: code * scale, rounded to float32."""
    v = np.float32(codes * np.asarray(scales, dtype=np.float64)[..., None]).astype(np.float64)
    return v.reshape(v.shape[:-2] + (-1,))[..., :inner]
