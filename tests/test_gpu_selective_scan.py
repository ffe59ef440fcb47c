"""The selective scan on the GPU (forward, backward, single-token step, autograd) against the
float64 definitions.

Tolerances, element by element, in steps e = 2^-24 of float32.  delta is off by Ed = e |raw|
sigmoid(raw) + (14 + 2 |raw|) e delta (the sum's rounding through the slope of the softplus; an
exponential of an argument |raw|, a reciprocal and a series); a decay a = exp(delta A) by a
((16 + 4 |delta A|) e + |A| Ed): the power of two 4 e, products 3 e, a share of the tile's
correction, which is formed with the same errors.  Every token multiplies and adds, a scan in
segments at most 60 roundings more on the way to a token.  With Hm the recurrence of the
magnitudes,
    Eh_t = a Eh_{t-1} + Ea (Hm_{t-1} + Eh_{t-1}) + Eb + 3 e Hm_t,  Eb = |u B| Ed + 4 e |b|,
plus 60 e Hm_t bounds a state's error, and the same in reverse time that of dh and g = a dh.
Products of both follow by the product rule.  Sums over N states have at most N + 8 roundings,
sums over channels 16 + D / 8, sums over tokens T + B + 40.  An output in bf16 is off by half a
step more, 2^-8 of its value (float32: 2^-24); 1e-34 stands for underflow."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as R
from constant_state_recurrence_gb300 import sanatan as S
from gpu_util import dev, f64
from test_gpu_layer_norm import BF16, E, F32, close

pytestmark = pytest.mark.gpu

NAMES = ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")


def make(b, T, D, N, dtype, seed, gated=True, h0=True, fast=False):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    size = torch.exp(torch.rand(D, generator=gen) * 4.6 - (2.3 if fast else 6.9))
    x = dict(u=n(b, T, D).to(dtype), dt=(0.6 * n(b, T, D)).to(dtype),
             A=-(torch.arange(N) + 1.0) * torch.exp(0.1 * n(D, N)), B=n(b, T, N).to(dtype),
             C=n(b, T, N).to(dtype), D=1 + 0.1 * n(D), z=n(b, T, D).to(dtype) if gated else None,
             dt_bias=size + torch.log(-torch.expm1(-size)), h0=0.5 * n(b, D, N) if h0 else None)
    return x, n(b, T, D).to(dtype), n(b, D, N) if h0 else None


def bounds(x, soft, lens, dy=None, dh=None):
    """Bounds before the outputs' own rounding, all in float64 from the definitions."""
    m = np.abs
    u, dt, A, B, C, D, z, bias, h0 = (x[k] for k in NAMES)
    b, T, W = u.shape
    N = A.shape[1]
    there = np.ones((b, T), bool) if lens is None else np.arange(T)[None] < np.asarray(lens)[:, None]
    th = there[..., None]
    raw = dt + (0 if bias is None else bias)
    delta = R.softplus(raw) if soft else raw
    Ed = E * m(raw) * R.sigmoid(raw) + (14 + 2 * m(raw)) * E * delta if soft else 2 * E * m(raw)
    delta, Ed = np.where(th, delta, 0.0), np.where(th, Ed, 0.0)
    u, B, C = (np.where(th, t, 0.0) for t in (u, B, C))
    md = m(delta)
    skip = 0 * u if D is None else np.broadcast_to(D, u.shape)
    a = np.exp(delta[..., None] * A)
    Ea = a * ((16 + 4 * m(delta[..., None] * A)) * E * th[..., None] + m(A) * Ed[..., None])
    bm = m((delta * u)[..., None] * B[:, :, None])
    Eb = m(u[..., None] * B[:, :, None]) * Ed[..., None] + 4 * E * bm
    Hm, Eh = np.zeros((b, T + 1, W, N)), np.zeros((b, T + 1, W, N))
    if h0 is not None:
        Hm[:, 0] = m(h0)
    for t in range(T):
        Hm[:, t + 1] = a[:, t] * Hm[:, t] + bm[:, t]
        Eh[:, t + 1] = a[:, t] * Eh[:, t] + Ea[:, t] * (Hm[:, t] + Eh[:, t]) + Eb[:, t] \
            + 3 * E * Hm[:, t + 1]
    Eh = Eh + 60 * E * Hm
    mC = m(C)[:, :, None]
    Ym = (mC * Hm[:, 1:]).sum(-1) + m(skip * u)
    Ey = (mC * Eh[:, 1:]).sum(-1) + (N + 8) * E * Ym
    gate = np.ones_like(u)
    kz = 0 * u
    if z is not None:
        z = np.where(th, z, 0.0)
        gate, kz = z * R.sigmoid(z), (12 + 2 * m(z)) * E
    out = dict(y=m(gate) * (Ey + kz * (Ym + Ey)), last=Eh[:, -1], marks=Eh[:, :-1][:, ::16])
    if dy is None:
        return out
    dy = np.where(th, dy, 0.0)
    v, Ev = dy * gate, kz * m(dy * gate)
    if z is not None:
        sg = R.sigmoid(z)
        two = m(sg) + m(z * sg * (1 - sg))
        out["dz"] = m(dy) * (m(R.silu_slope(z)) * Ey + (24 + 4 * m(z)) * E * two * (Ym + Ey))
    g = np.zeros((b, W, N)) if dh is None else m(dh)
    eg = np.zeros((b, W, N))
    Dm, Edh, Gm, Eg = (np.zeros((b, T, W, N)) for _ in range(4))
    for t in range(T - 1, -1, -1):
        Dm[:, t] = g + m(v[:, t])[..., None] * mC[:, t]
        Edh[:, t] = eg + Ev[:, t][..., None] * mC[:, t] + 3 * E * Dm[:, t]
        g = a[:, t] * Dm[:, t]
        eg = a[:, t] * Edh[:, t] + Ea[:, t] * (Dm[:, t] + Edh[:, t]) + E * g
        Gm[:, t], Eg[:, t] = g, eg
    Edh, Eg = Edh + 60 * E * Dm, Eg + 60 * E * Gm
    out["dh0"] = Eg[:, 0] if T else eg
    Hb, Eb_ = Hm[:, :-1], Eh[:, :-1]
    Wm = Gm * Hb
    Ew = Gm * Eb_ + Eg * Hb + Eg * Eb_ + 2 * E * Wm
    mB = m(B)[:, :, None]
    sB, EsB = (mB * Dm).sum(-1), (mB * Edh).sum(-1) + (N + 8) * E * (mB * Dm).sum(-1)
    sA = (m(A) * Wm).sum(-1)
    EsA = (m(A) * Ew).sum(-1) + (N + 10) * E * sA
    out["du"] = md * EsB + Ed * (sB + EsB) + m(skip) * Ev + 4 * E * (md * sB + m(skip * v))
    ed = m(u) * EsB + EsA + 4 * E * (m(u) * sB + sA)
    top = m(u) * sB + sA
    slope, ks = (R.sigmoid(raw), (12 + 2 * m(raw)) * E) if soft else (np.ones_like(raw), 0 * raw)
    out["ddt"] = np.where(th, slope * (ed + ks * (top + ed) + E * m(raw) * top), 0.0)
    n = (T + b + 40) * E
    d4, e4 = md[..., None], Ed[..., None]
    out["dA"] = (d4 * Ew + e4 * (Wm + Ew)).sum((0, 1)) + n * (d4 * Wm).sum((0, 1))
    out["ddt_bias"] = out["ddt"].sum((0, 1)) + n * np.where(th, slope * top, 0.0).sum((0, 1))
    out["dD"] = (Ev * m(u)).sum((0, 1)) + n * m(v * u).sum((0, 1))
    ch = (16 + W / 8) * E
    du = m(delta * u)[..., None]
    edu = (Ed * m(u))[..., None] + E * du
    out["dB"] = (du * Edh + edu * (Dm + Edh)).sum(2) + ch * (du * Dm).sum(2)
    mv, ev = m(v)[..., None], Ev[..., None]
    out["dC"] = (mv * Eh[:, 1:] + ev * (Hm[:, 1:] + Eh[:, 1:])).sum(2) + ch * (mv * Hm[:, 1:]).sum(2)
    return out


def on(x, place=lambda t: t.to(dev())):
    return {k: None if t is None else place(t) for k, t in x.items()}


def run(x, dy, dh, soft=True, lens=None, place=lambda t: t.to(dev())):
    """(forward's outputs, gradients) on the device."""
    d = on(x, place)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int64).to(dev())
    h0 = d.pop("h0")
    y, h, marks = S.sanatan_selective_scan_fwd(**d, softplus=soft, h0=h0, lens=ln,
                                               want_state=True, want_marks=True)
    g = S.sanatan_selective_scan_bwd(**d, dy=place(dy), marks=marks, softplus=soft, lens=ln,
                                     dh_last=None if dh is None else place(dh), want_dh0=True)
    torch.cuda.synchronize()
    return (y, h, marks), g


def check(b, T, D, N, dtype, soft=True, gated=True, h0=True, lens=None, seed=0, fast=False,
          drop=(), place=lambda t: t.to(dev())):
    x, dy, dh = make(b, T, D, N, dtype, seed, gated, h0, fast)
    for k in drop:
        x[k] = None
    if not soft:
        x["dt"], x["dt_bias"] = (0.1 * x["dt"].float().abs()).to(dtype), None
    (y, h, marks), g = run(x, dy, dh, soft, lens, place)
    n = {k: None if t is None else f64(t) for k, t in x.items()}
    cut = None if lens is None else R.lengths(lens, b, T)
    args = dict(n, soft=soft, lens=cut)
    y_ref, h_ref, before = R.selective_scan(**args)
    ref = R.selective_scan_backward(**args, dy=f64(dy), dh_last=None if dh is None else f64(dh))
    bd = bounds(n, soft, cut, f64(dy), None if dh is None else f64(dh))
    there = np.ones((b, T, 1)) if cut is None else \
        (np.arange(T)[None] < np.asarray(cut)[:, None])[..., None]
    close(y, y_ref, bd["y"] * there + 1e-34, dtype, "y")
    close(h, h_ref, bd["last"] + 1e-34, F32, "h_last")
    real = there[:, ::16, 0].astype(bool)   # a mark is written where its tile has a token
    close(marks[torch.from_numpy(real).to(dev())], before[:, ::16][real],
          bd["marks"][real] + 1e-34, F32, "marks")
    for k, ty in (("du", dtype), ("ddt", dtype), ("dz", dtype), ("dA", F32), ("dB", dtype),
                  ("dC", dtype), ("dD", F32), ("ddt_bias", F32), ("dh0", F32)):
        if g[k] is None:
            assert {"dz": "z", "dD": "D", "ddt_bias": "dt_bias"}[k] and x[
                {"dz": "z", "dD": "D", "ddt_bias": "dt_bias"}[k]] is None, k
            continue
        close(g[k], ref[k], bd[k] + 1e-34, ty, k)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,T,D,N", [
    (1, 1, 1, 1), (1, 2, 3, 2), (2, 5, 8, 4), (1, 15, 32, 16), (2, 16, 33, 16), (1, 17, 31, 16),
    (3, 33, 40, 16), (2, 50, 130, 3), (1, 40, 7, 13), (2, 20, 24, 8), (1, 64, 9, 5),
    (1, 35, 16, 32), (2, 18, 5, 17), (1, 33, 6, 64), (1, 20, 3, 50), (1, 19, 4, 128),
    (1, 17, 2, 99), (9, 3, 64, 16), (1, 70, 5, 16), (2, 66, 8, 64),
    (1, 70, 4, 128), (2, 90, 3, 100)])
def test_against_the_definition(b, T, D, N, dtype):
    check(b, T, D, N, dtype, seed=T + D + N, h0=T % 2 == 1, gated=(T + D) % 3 != 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,T,D,N", [(1, 300, 8, 16), (2, 131, 16, 4), (1, 450, 5, 9),
                                     (3, 200, 32, 16), (1, 130, 3, 40)])
def test_sequences_cut_into_segments(b, T, D, N, dtype):
    """Few channels and many tokens: the three-kernel forms, both directions."""
    assert S.selective_scan_fwd_workspace_size(b, T, D, N) > 0
    check(b, T, D, N, dtype, seed=T, lens=[T - 37, T, 70][:b])


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("N,D", [(16, 40), (6, 9), (1, 33)])
def test_lengths(N, D, fast):
    """From no token to all, on both sides of a tile's border, values outside [0, T]."""
    check(8, 50, D, N, F32, lens=[0, 1, 15, 16, 17, 50, -3, 99], seed=N, fast=fast)


@pytest.mark.parametrize("drop", [("D",), ("dt_bias",), ("D", "z", "dt_bias")])
@pytest.mark.parametrize("soft", [True, False])
def test_without_parts(drop, soft):
    check(2, 35, 40, 16, F32, soft=soft, drop=drop, seed=3)
    check(1, 150, 8, 8, BF16, soft=soft, drop=drop, seed=4)


@pytest.mark.parametrize("dtype,N", [(F32, 16), (BF16, 16), (BF16, 8), (F32, 5)])
def test_parts_of_larger_tensors(dtype, N):
    """Addresses at any element, and states, too."""
    def place(t):
        big = torch.zeros(t.numel() + 1, dtype=t.dtype, device=dev())
        big[1:].copy_(t.flatten())
        return big[1:].view(t.shape)
    check(2, 37, 40, N, dtype, place=place, seed=5)


@pytest.mark.parametrize("dtype,D,N,pad", [(F32, 32, 16, 8), (BF16, 48, 16, 8), (BF16, 33, 7, 3)])
def test_rows_of_wider_projections(dtype, D, N, pad):
    """B, C and z out of wider rows give what dense ones give."""
    x, dy, dh = make(2, 45, D, N, dtype, 6)
    want, gw = run(x, dy, dh)
    rows = torch.randn(2, 45, pad + 2 * N).to(dtype).to(dev())
    both = torch.randn(2, 45, 2 * D).to(dtype).to(dev())
    d = on(x)
    rows[..., pad:pad + N], rows[..., pad + N:], both[..., D:] = d["B"], d["C"], d["z"]
    d.update(B=rows[..., pad:pad + N], C=rows[..., pad + N:], z=both[..., D:])
    h0 = d.pop("h0")
    y, h, marks = S.sanatan_selective_scan_fwd(**d, h0=h0, want_state=True, want_marks=True)
    g = S.sanatan_selective_scan_bwd(**d, dy=dy.to(dev()), marks=marks, dh_last=dh.to(dev()),
                                     want_dh0=True)
    assert all(torch.equal(p, q) for p, q in zip((y, h, marks), want))
    assert all(torch.equal(g[k], gw[k]) for k in g)


def test_no_tokens_and_no_sequences():
    x, dy, dh = make(2, 0, 12, 16, F32, 7)
    (y, h, _), g = run(x, dy, dh)
    assert y.shape == (2, 0, 12) and torch.equal(h.cpu(), x["h0"])
    assert torch.equal(g["dh0"].cpu(), dh)
    assert not any(g[k].any() for k in ("dA", "dD", "ddt_bias"))
    x, dy, dh = make(0, 5, 12, 16, F32, 7)
    _, g = run(x, dy, dh)
    assert not any(g[k].any() for k in ("dA", "dD", "ddt_bias"))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_channels(dtype):
    """dB and dC are sums over channels: zeros, written whole."""
    x, dy, dh = make(2, 5, 0, 16, dtype, 7)
    left = torch.full((2, 2, 5, 16), float("nan"), dtype=dtype, device=dev())
    del left   # (what the outputs may be allocated on)
    (y, h, _), g = run(x, dy, dh)
    assert y.shape == (2, 5, 0) and h.shape == (2, 0, 16)
    assert g["dB"].shape == g["dC"].shape == (2, 5, 16)
    assert torch.equal(g["dB"], torch.zeros_like(g["dB"]))
    assert torch.equal(g["dC"], torch.zeros_like(g["dC"]))


def test_the_same_bits_and_states_in_place():
    for b, T, D, N in ((1, 400, 24, 16), (3, 40, 100, 16), (1, 300, 3, 6)):
        x, dy, dh = make(b, T, D, N, F32, T)
        (y, h, marks), g = run(x, dy, dh)
        for _ in range(2):
            (y2, h2, m2), g2 = run(x, dy, dh)
            assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(marks, m2)
            assert all(torch.equal(g[k], g2[k]) for k in g)
        d = on(x)
        state = d.pop("h0").clone()
        y3, _, _ = S.sanatan_selective_scan_fwd(**d, h0=state, h_out=state)
        assert torch.equal(y, y3) and torch.equal(h, state)


def test_what_is_behind_a_sequence_is_not_read():
    for T, D, N, dtype in ((40, 36, 16, F32), (300, 8, 16, BF16), (30, 7, 5, BF16)):
        x, dy, dh = make(2, T, D, N, dtype, 8)
        lens = [T - 9, 0]
        want, gw = run(x, dy, dh, lens=lens)
        for t in [x[k] for k in ("u", "dt", "B", "C", "z")] + [dy]:
            t[0, T - 9:] = float("nan")
            t[1] = float("inf")
        got, g = run(x, dy, dh, lens=lens)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        assert all(torch.equal(g[k], gw[k]) for k in g)


def test_what_is_not_finite_stays_in_its_sequence_and_channel():
    x, dy, dh = make(2, 60, 40, 16, F32, 9)
    (y, h, _), _ = run(x, dy, dh)
    x["u"][1, 20, 7] = float("nan")
    (y2, h2, _), _ = run(x, dy, dh)
    hit = torch.zeros(2, 60, 40, dtype=torch.bool)
    hit[1, 20:, 7] = True
    hit = hit.to(dev())
    assert torch.equal(y[~hit], y2[~hit]) and y2[hit].isnan().all() and h2[1, 7].isnan().all()


def test_decays_of_every_size():
    """Steps from far below the rounding of 1 to what leaves no memory: delta A from 1e-9 to
    200, also without any decay."""
    x, dy, dh = make(1, 60, 48, 16, F32, 10)
    x["dt_bias"] = torch.linspace(-18, 5, 48)
    x["A"][3] = 0.0
    (y, h, _), g = run(x, dy, dh)
    n = {k: f64(t) for k, t in x.items()}
    bd = bounds(n, True, None, f64(dy), f64(dh))
    y_ref, h_ref, _ = R.selective_scan(**n)
    close(y, y_ref, bd["y"] + 1e-34, F32, "y")
    close(h, h_ref, bd["last"] + 1e-34, F32, "h")
    ref = R.selective_scan_backward(**n, dy=f64(dy), dh_last=f64(dh))
    for k in ("du", "ddt", "dA", "dB", "dC", "dh0"):
        close(g[k], ref[k], bd[k] + 1e-34, F32, k)


def test_a_long_memory_does_not_gather_the_decays_errors():
    """Constant steps, memories of 100 to 100000 tokens, 4000 tokens: the state within 4e-6 of
    its value.  (With the decays' mean error of 0.1 to 0.4 steps of 2^-24 it would be off by up
    to that times the smaller of memory and tokens, 1e-5 and more.)  What is allowed is the
    rounding of delta, the same for every token, 2^-24 and the softplus's 8 e of delta: relative
    to the state at most twice that, 1e-6, and of A log2(e); roundings of the state itself
    are 0.3 e sqrt(tokens) = 1.1e-6."""
    T, D = 4000, 16
    delta = torch.logspace(-5, -2, D)
    u, one = torch.ones(1, T, D), torch.ones(1, T, 1)
    for pieces in (1, 7):
        h = None
        for part in range(pieces):
            at = slice(part * T // pieces, (part + 1) * T // pieces)
            d = [t[:, at].contiguous().to(dev()) for t in (u, one)]
            _, h, _ = S.sanatan_selective_scan_fwd(
                d[0], (0 * d[0]).contiguous(), -torch.ones(D, 1, device=dev()), d[1], d[1],
                dt_bias=torch.log(torch.expm1(delta)).to(dev()), h0=h, want_state=True)
        exact = np.log1p(np.exp(f64(torch.log(torch.expm1(delta)))))
        want = exact * -np.expm1(-T * exact) / -np.expm1(-exact)
        assert np.abs(f64(h)[0, :, 0] / want - 1).max() <= 4e-6


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,D,N,gated", [(1, 1, 1, True), (1, 64, 16, True), (7, 33, 16, False),
                                         (5, 40, 5, True), (2, 9, 100, True), (300, 24, 8, True)])
def test_single_tokens(b, D, N, gated, dtype):
    x, _, _ = make(b, 3, D, N, dtype, b + D, gated)
    d = on(x)
    h = d.pop("h0").clone()
    n = {k: None if t is None else f64(t) for k, t in x.items()}
    y_ref, h_ref, _ = R.selective_scan(**n)
    bd = bounds(n, True, None)
    for t in range(3):
        one = {k: v[:, t] if v is not None and v.dim() == 3 else v for k, v in d.items()}
        one.update(u=one["u"].contiguous(), dt=one["dt"].contiguous())
        y = S.sanatan_selective_scan_step(h, **one)
        close(y, y_ref[:, t], bd["y"][:, t], dtype, "y")
    close(h, h_ref, bd["last"], F32, "h")


def test_autograd_against_the_formula_and_differences():
    x, dy, dh = make(2, 30, 12, 6, F32, 11)
    d = on(x)
    leaves = [d[k].clone().requires_grad_() for k in NAMES]
    u, dt, A, B, C, D, z, bias, h0 = leaves
    y, h = S.SelectiveScan.apply(u, dt, A, B, C, D, z, bias, True, h0)
    ((y * dy.to(dev())).sum() + (h * dh.to(dev())).sum()).backward()
    n = {k: f64(t) for k, t in x.items()}
    ref = R.selective_scan_backward(**n, dy=f64(dy), dh_last=f64(dh))
    bd = bounds(n, True, None, f64(dy), f64(dh))
    rng = np.random.default_rng(12)
    way = {k: rng.standard_normal(n[k].shape) for k in NAMES}
    got = room = 0.0
    for k, leaf in zip(NAMES, leaves):
        close(leaf.grad, ref["d" + k], bd["d" + k] + 1e-34, F32, k)
        got += (f64(leaf.grad) * way[k]).sum()
        room += (np.abs(way[k]) * (bd["d" + k] + E * np.abs(ref["d" + k]))).sum()

    def loss(sign):
        y, h, _ = R.selective_scan(**{k: n[k] + sign * 1e-5 * way[k] for k in NAMES})
        return (y * f64(dy)).sum() + (h * f64(dh)).sum()

    diff = (loss(1) - loss(-1)) / 2e-5
    assert abs(got - diff) <= room + 1e-6 * abs(diff)


def test_autograd_with_one_of_the_outputs_only():
    x, dy, dh = make(1, 20, 8, 4, F32, 13)
    d = on(x)
    u = d["u"].requires_grad_()
    rest = [d[k] for k in ("dt", "A", "B", "C", "D")]
    _, h = S.SelectiveScan.apply(u, *rest)
    h.sum().backward()
    a, u.grad = u.grad.clone(), None
    y, _ = S.SelectiveScan.apply(u, *rest)
    y[:, 3].sum().backward()
    assert a.any() and u.grad[:, :4].any() and not u.grad[:, 4:].any()


def test_captured_training_step_and_token():
    for b, T, D, N in ((2, 90, 72, 16), (1, 400, 16, 16)):
        x, dy, dh = make(b, T, D, N, BF16, 14)
        d, dyd = on(x), dy.to(dev())
        h0 = d.pop("h0")
        state = h0.clone()
        one = {k: v[:, 0].contiguous() if v.dim() == 3 else v for k, v in d.items()}

        def step():
            y, h, marks = S.sanatan_selective_scan_fwd(**d, h0=h0, want_state=True,
                                                       want_marks=True)
            g = S.sanatan_selective_scan_bwd(**d, dy=dyd, marks=marks, want_dh0=True)
            return [y, h] + list(g.values())

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            there = step()
            S.sanatan_selective_scan_step(state, **one)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(there, step()))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
            tok = S.sanatan_selective_scan_step(state, **one)
        d["u"].mul_(-0.5)
        state.copy_(h0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step()))
        again = h0.clone()
        assert torch.equal(tok, S.sanatan_selective_scan_step(again, **one))
        assert torch.equal(state, again)


def test_refusals():
    x, dy, dh = make(2, 9, 16, 4, F32, 15)
    d = on(x)
    h0 = d.pop("h0")
    f = S.sanatan_selective_scan_fwd
    for bad in (lambda: f(**{**d, "A": torch.ones(16, 129, device=dev())}),
                lambda: f(**{**d, "A": d["A"].bfloat16()}),
                lambda: f(**{**d, "dt": d["dt"].bfloat16()}),
                lambda: f(**{**d, "u": d["u"].half(), "dt": d["dt"].half()}),
                lambda: f(**{**d, "B": d["B"][..., :3]}),
                lambda: f(**{**d, "B": d["B"][..., :1].expand(2, 9, 4)}),
                lambda: f(**{**d, "z": d["z"].transpose(1, 2)}),
                lambda: f(**{**d, "u": d["u"].transpose(0, 1), "dt": d["dt"].transpose(0, 1)}),
                lambda: f(**d, h0=h0[:1]),
                lambda: f(**d, lens=torch.ones(2, dtype=torch.int32, device=dev())),
                lambda: S.sanatan_selective_scan_bwd(
                    **d, dy=dy.to(dev()), marks=torch.ones(2, 2, 16, 4, device=dev())),
                lambda: S.sanatan_selective_scan_step(h0, **d)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(S.SanatanError):
        f(**d, out=d["u"])
