"""The gated linear recurrence on the GPU (scan forward, backward, single-token
step, autograd) against the float64 definitions.

Tolerances, element by element, from the rounding steps e = 2^-24 of float32: a
decay and its 1 - a are within k = (10 + 2 |g|) e of their values (exponential
2 ulp, its argument's product half an ulp of |g|, sum and reciprocal 1 ulp each);
every token adds a multiplication and an addition, and a scan in pieces at most
40 more additions on the way to a token.  With Hm the recurrence of |u| and |h0|,
    E_t = a_t (E_{t-1} + (k + 3 e) Hm_{t-1}) + (k + 3 e) |u_t|
bounds the state's error up to 40 e Hm_t, and the same in reverse time bounds
dh's.  Products of both add up.  An output in bf16 is off by half a step more,
2^-8 of its value (float32: 2^-24); 1e-36 stands for underflow."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.state_oracle as R
from constant_state_recurrence_gb300 import sanatan as S
from gpu_util import dev, f64

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


def make(B, T, D, dtype, gate, seed, h0=True, bias=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, D, generator=gen)
    g = torch.randn(B, T, D, generator=gen) + bias
    if gate == "log":
        g = -torch.nn.functional.softplus(-g)
    dy = torch.randn(B, T, D, generator=gen)
    h = torch.randn(B, D, generator=gen) if h0 else None
    dh = torch.randn(B, D, generator=gen) if h0 else None
    return x.to(dtype), g.to(dtype), dy.to(dtype), h, dh


def bounds(x, g, gate, h0, dy=None, dh_last=None, lens=None):
    """Error bounds before the outputs' own rounding: dict of arrays."""
    B, T, D = x.shape
    a, keep, u = R.gates(x, g, gate)
    k = (10 + 2 * np.where(np.isfinite(g), np.abs(g), 0.0)) * E
    if lens is not None:
        gone = (np.arange(T)[None] >= np.asarray(lens)[:, None])[..., None]
        a, u, k = np.where(gone, 1.0, a), np.where(gone, 0.0, u), np.where(gone, 0.0, k)
    Hm = np.zeros((B, T + 1, D))
    Er = np.zeros((B, T + 1, D))
    if h0 is not None:
        Hm[:, 0] = np.abs(h0)
    for t in range(T):
        Hm[:, t + 1] = a[:, t] * Hm[:, t] + np.abs(u[:, t])
        Er[:, t + 1] = a[:, t] * (Er[:, t] + (k[:, t] + 3 * E) * Hm[:, t]) \
            + (k[:, t] + 3 * E) * np.abs(u[:, t])
    Er = Er + 40 * E * Hm + 1e-36
    out = dict(y=Er[:, 1:], last=Er[:, -1], before=Er[:, :-1])
    if dy is None:
        return out
    Dm, Ed = np.zeros((B, T, D)), np.zeros((B, T, D))
    m = np.zeros((B, D)) if dh_last is None else np.abs(dh_last)
    e = np.zeros((B, D))
    for t in range(T - 1, -1, -1):
        Dm[:, t] = m + np.abs(dy[:, t])
        Ed[:, t] = e + 2 * E * Dm[:, t]
        e = a[:, t] * (Ed[:, t] + (k[:, t] + 3 * E) * Dm[:, t])
        m = a[:, t] * Dm[:, t]
    Ed = Ed + 40 * E * Dm + 1e-36
    out["dh0"] = e + 40 * E * m + 1e-36
    Hb, Eb = Hm[:, :-1], Er[:, :-1]
    if gate == "log":
        out["dx"] = Ed
        out["dg"] = a * (Hb * Ed + Dm * Eb) + (k + 4 * E) * a * Dm * Hb
    else:
        w = Hb + np.abs(x)
        out["dx"] = keep * (Ed + (k + 2 * E) * Dm)
        out["dg"] = a * keep * (w * Ed + Dm * (Eb + 2 * E * w)) \
            + (2 * k + 6 * E) * a * keep * Dm * w
    return out


def close(got, ref, bound, dtype, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    room = bound * (1 + 1e-3) + HALF[dtype] * (np.abs(ref) + bound) + 1e-36
    off = np.abs(got - ref) - room
    assert np.isfinite(got).all(), what
    assert off.max(initial=-1.0) <= 0, (what, np.unravel_index(off.argmax(), off.shape), off.max())


def check(B, T, D, dtype, gate, seed=0, h0=True, lens=None, bias=1.0):
    x, g, dy, h, dh = make(B, T, D, dtype, gate, seed, h0, bias)
    d = lambda t: None if t is None else t.to(dev())  # noqa: E731
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int64)
    y, last, marks = S.sanatan_gated_scan_fwd(d(x), d(g), gate, h0=d(h), lens=d(ln),
                                              want_state=True, want_marks=True)
    gr = S.sanatan_gated_scan_bwd(d(x), d(g), d(dy), marks, gate, lens=d(ln), dh_last=d(dh),
                                  want_dh0=True)
    S.device_status()
    n = lambda t: None if t is None else f64(t)  # noqa: E731
    cut = None if lens is None else [min(max(v, 0), T) for v in lens]
    y_ref, last_ref, before = R.gated_scan(n(x), n(g), gate, n(h), cut)
    dx, dg, dh0 = R.gated_scan_backward(n(x), n(g), gate, n(dy), n(h), cut, n(dh))
    b = bounds(n(x), n(g), gate, n(h), n(dy), n(dh), cut)
    there = np.ones((B, T, 1)) if cut is None else \
        (np.arange(T)[None] < np.asarray(cut)[:, None])[..., None]
    close(y, y_ref, b["y"] * there, dtype, "y")
    close(last, last_ref, b["last"], F32, "h_last")
    close(marks, before[:, ::64], b["before"][:, ::64], F32, "marks")
    close(gr["dx"], dx, b["dx"] * there, dtype, "dx")
    close(gr["dg"], dg, b["dg"] * there, dtype, "dg")
    close(gr["dh0"], dh0, b["dh0"], F32, "dh0")


SHAPES = [(1, 1, 1), (1, 1, 64), (2, 2, 3), (1, 7, 4), (3, 63, 65), (2, 64, 64), (2, 65, 130),
          (1, 127, 768), (2, 128, 12), (3, 129, 100), (1, 1000, 33), (5, 300, 257), (70, 5, 64),
          (2, 2049, 72), (400, 9, 65), (330, 70, 64)]


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_forward_and_backward(B, T, D, dtype, gate):
    check(B, T, D, dtype, gate, seed=B + T + D)


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("B,T,D,lens", [
    (4, 150, 64, [150, 149, 1, 0]), (3, 700, 70, [650, 64, 128]), (2, 40, 5, [-7, 1 << 40]),
    (1, 2000, 8, [1030])])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lengths(B, T, D, lens, gate, dtype):
    check(B, T, D, dtype, gate, seed=T, lens=lens)


@pytest.mark.parametrize("D", [66, 64])
def test_lengths_keep_out_what_lies_behind(D):
    """NaN in the padding reaches neither outputs, state nor gradients."""
    x, g, dy, h, _ = make(2, 200, D, F32, "sigmoid", 3)
    lens = torch.tensor([130, 3], dtype=torch.int64)
    for b in range(2):
        for t in (x, g, dy):
            t[b, lens[b]:] = float("nan")
    d = lambda t: t.to(dev())  # noqa: E731
    y, last, marks = S.sanatan_gated_scan_fwd(d(x), d(g), "sigmoid", h0=d(h), lens=d(lens),
                                              want_state=True, want_marks=True)
    gr = S.sanatan_gated_scan_bwd(d(x), d(g), d(dy), marks, "sigmoid", lens=d(lens), want_dh0=True)
    for b in range(2):
        n = int(lens[b])
        for t in (y, gr["dx"], gr["dg"]):
            assert not t[b, n:].any() and torch.isfinite(t[b]).all()
    assert torch.isfinite(last).all() and torch.isfinite(gr["dh0"]).all()


def test_without_initial_state_and_without_gradients_of_it():
    check(2, 130, 48, BF16, "log", seed=4, h0=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_memory(dtype):
    """Decays next to 1 over a long sequence (a channel's memory: hundreds of tokens)."""
    check(1, 6000, 16, dtype, "log", seed=9, bias=6.0)
    check(1, 6000, 16, dtype, "sigmoid", seed=10, bias=6.0)


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
def test_closed_and_open_gates(gate):
    """Gates of -inf start a new text; the sigmoid's of +inf keep the state."""
    x, g, dy, h, dh = make(1, 300, 64, F32, gate, 11)
    g[0, 100] = g[0, 228, :32] = -float("inf")
    if gate == "sigmoid":
        g[0, 50] = float("inf")
    d = lambda t: t.to(dev())  # noqa: E731
    y, last, marks = S.sanatan_gated_scan_fwd(d(x), d(g), gate, h0=d(h), want_state=True,
                                              want_marks=True)
    gr = S.sanatan_gated_scan_bwd(d(x), d(g), d(dy), marks, gate, dh_last=d(dh), want_dh0=True)
    y_ref, _, _ = R.gated_scan(f64(x), f64(g), gate, f64(h))
    dx, dg, dh0 = R.gated_scan_backward(f64(x), f64(g), gate, f64(dy), f64(h), None, f64(dh))
    b = bounds(f64(x), f64(g), gate, f64(h), f64(dy), f64(dh))
    close(y, y_ref, b["y"], F32, "y")
    close(gr["dx"], dx, b["dx"], F32, "dx")
    close(gr["dg"], dg, b["dg"], F32, "dg")
    close(gr["dh0"], dh0, b["dh0"], F32, "dh0")
    if gate == "log":       # a = 0: nothing of what lies before, to the bit
        assert torch.equal(y[:, 100], d(x)[:, 100]) and not gr["dg"][:, 100].any()


def test_values_that_are_not_finite_stay_in_their_channel():
    x, g, _, _, _ = make(2, 500, 70, F32, "log", 12)
    x[0, 200, 7] = float("nan")
    x[1, 300, 69] = float("inf")
    y, last, _ = S.sanatan_gated_scan_fwd(x.to(dev()), g.to(dev()), want_state=True)
    bad = ~torch.isfinite(y).cpu()
    want = torch.zeros_like(bad)
    want[0, 200:, 7] = True
    want[1, 300:, 69] = True
    assert torch.equal(bad, want)
    assert torch.isnan(last[0, 7]) and torch.isinf(last[1, 69])


def test_one_call_is_two_halves():
    """The state carries a sequence over two calls, and its gradient back."""
    x, g, dy, h, dh = make(2, 333, 96, F32, "log", 13)
    d = lambda t: t.contiguous().to(dev())  # noqa: E731
    whole, last, _ = S.sanatan_gated_scan_fwd(d(x), d(g), h0=d(h), want_state=True)
    y1, s1, m1 = S.sanatan_gated_scan_fwd(d(x[:, :200]), d(g[:, :200]), h0=d(h), want_state=True,
                                          want_marks=True)
    y2, s2, m2 = S.sanatan_gated_scan_fwd(d(x[:, 200:]), d(g[:, 200:]), h0=s1, want_state=True,
                                          want_marks=True)
    b = bounds(f64(x), f64(g), "log", f64(h), f64(dy), f64(dh))
    assert (np.abs(f64(torch.cat([y1, y2], 1)) - f64(whole)) <= 2 * b["y"]).all()
    assert (np.abs(f64(s2) - f64(last)) <= 2 * b["last"]).all()
    g2 = S.sanatan_gated_scan_bwd(d(x[:, 200:]), d(g[:, 200:]), d(dy[:, 200:]), m2, dh_last=d(dh),
                                  want_dh0=True)
    g1 = S.sanatan_gated_scan_bwd(d(x[:, :200]), d(g[:, :200]), d(dy[:, :200]), m1,
                                  dh_last=g2["dh0"], want_dh0=True)
    dx, dg, dh0 = R.gated_scan_backward(f64(x), f64(g), "log", f64(dy), f64(h), None, f64(dh))
    close(torch.cat([g1["dx"], g2["dx"]], 1), dx, 2 * b["dx"], F32, "dx")
    close(torch.cat([g1["dg"], g2["dg"]], 1), dg, 2 * b["dg"], F32, "dg")
    close(g1["dh0"], dh0, 2 * b["dh0"], F32, "dh0")


def test_same_call_same_bits():
    x, g, dy, h, dh = (t.to(dev()) for t in make(2, 1500, 200, BF16, "sigmoid", 14))
    runs = []
    for _ in range(3):
        y, last, marks = S.sanatan_gated_scan_fwd(x, g, "sigmoid", h0=h, want_state=True,
                                                  want_marks=True)
        gr = S.sanatan_gated_scan_bwd(x, g, dy, marks, "sigmoid", dh_last=dh, want_dh0=True)
        runs.append((y, last, marks, gr["dx"], gr["dg"], gr["dh0"]))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,D", [(1, 1), (1, 768), (3, 5), (9, 129), (400, 768)])
def test_step(N, D, dtype, gate):
    x, g, _, h, _ = make(N, 1, D, dtype, gate, N + D)
    hd = h.to(dev())
    y = S.sanatan_gated_scan_step(hd, x[:, 0].contiguous().to(dev()),
                                  g[:, 0].contiguous().to(dev()), gate)
    ref = R.gated_scan_step(f64(h), f64(x[:, 0]), f64(g[:, 0]), gate)
    b = bounds(f64(x), f64(g), gate, f64(h))["last"]
    close(hd, ref, b, F32, "h")
    close(y, ref, b, dtype, "y")
    assert torch.equal(y, hd.to(dtype))


def test_steps_continue_a_scan():
    x, g, _, h, _ = make(3, 40, 100, F32, "sigmoid", 15)
    d = lambda t: t.contiguous().to(dev())  # noqa: E731
    _, state, _ = S.sanatan_gated_scan_fwd(d(x[:, :30]), d(g[:, :30]), "sigmoid", h0=d(h),
                                           want_state=True)
    ref, last, _ = R.gated_scan(f64(x), f64(g), "sigmoid", f64(h))
    b = bounds(f64(x), f64(g), "sigmoid", f64(h))
    for t in range(30, 40):
        y = S.sanatan_gated_scan_step(state, d(x[:, t]), d(g[:, t]), "sigmoid")
        close(y, ref[:, t], b["y"][:, t], F32, t)
    close(state, last, b["last"], F32, "state")


def test_empty_problems():
    h = torch.randn(2, 8, device=dev())
    x = torch.empty(2, 0, 8, device=dev())
    y, last, marks = S.sanatan_gated_scan_fwd(x, x, h0=h, want_state=True, want_marks=True)
    assert y.shape == x.shape and torch.equal(last, h) and marks.shape == (2, 0, 8)
    gr = S.sanatan_gated_scan_bwd(x, x, x, marks, dh_last=h, want_dh0=True)
    assert torch.equal(gr["dh0"], h)
    _, last, _ = S.sanatan_gated_scan_fwd(x, x, want_state=True)
    assert not last.any()
    for shape in ((0, 5, 8), (3, 5, 0)):
        x = torch.empty(shape, device=dev())
        y, last, _ = S.sanatan_gated_scan_fwd(x, x, want_state=True)
        assert y.shape == x.shape and last.shape == (shape[0], shape[2])
    e = torch.empty(0, 8, device=dev())
    assert S.sanatan_gated_scan_step(e, e, e).shape == (0, 8)


def test_large_sequence_sampled_channels():
    """B=1, T=32768, D=768 bf16 (a long prefill of a layer): every token of some
    channels, in every block of channels."""
    gen = torch.Generator(device=dev()).manual_seed(16)
    x = torch.randn(1, 32768, 768, generator=gen, device=dev()).to(BF16)
    g = (torch.randn(1, 32768, 768, generator=gen, device=dev()) + 2).to(BF16)
    y, last, _ = S.sanatan_gated_scan_fwd(x, g, "sigmoid", want_state=True)
    pick = torch.arange(0, 768, 31, device=dev())
    xs, gs = f64(x[..., pick]), f64(g[..., pick])
    ref, last_ref, _ = R.gated_scan(xs, gs, "sigmoid")
    b = bounds(xs, gs, "sigmoid", None)
    close(y[..., pick], ref, b["y"], BF16, "y")
    close(last[..., pick], last_ref, b["last"], F32, "last")


def test_offsets_beyond_32_bits():
    """B T D of more than 2^31 elements: the last sequence is where it should be."""
    B, T, D = 3, 32768, 22000
    x = torch.zeros(B, T, D, dtype=BF16, device=dev())
    g = torch.zeros(B, T, D, dtype=BF16, device=dev())
    x[2, -1] = torch.arange(D, device=dev()).remainder(251).to(BF16)
    x[2, -2] = 1.0
    y, last, _ = S.sanatan_gated_scan_fwd(x, g, want_state=True)     # a = 1: running sums
    want = torch.arange(D, device=dev()).remainder(251).float() + 1
    assert torch.equal(last[2], want) and not last[:2].any()
    assert torch.equal(y[2, -1], want.to(BF16)) and not y[:2].any() and not y[2, :-2].any()


def test_autograd_trains_gates_inputs_and_states():
    """Gradients through GatedScan of a projection shared by two scans, against
    float64 autograd-free formulas and differences of the float64 definition."""
    x, g, dy, h, dh = make(2, 70, 24, F32, "sigmoid", 17)
    xs = x.to(dev()).requires_grad_()
    gs = g.to(dev()).requires_grad_()
    h0 = h[:1].to(dev()).requires_grad_()          # one learned state for the whole batch
    y, last = S.GatedScan.apply(xs, gs, "sigmoid", h0.expand(2, -1).contiguous())
    (y * dy.to(dev())).sum().add((last * dh.to(dev())).sum()).backward()
    h2 = np.repeat(f64(h[:1]), 2, 0)
    dx, dg, dh0 = R.gated_scan_backward(f64(x), f64(g), "sigmoid", f64(dy), h2, None, f64(dh))
    b = bounds(f64(x), f64(g), "sigmoid", h2, f64(dy), f64(dh))
    close(xs.grad, dx, b["dx"], F32, "dx")
    close(gs.grad, dg, b["dg"], F32, "dg")
    close(h0.grad, dh0.sum(0, keepdims=True), b["dh0"].sum(0, keepdims=True), F32, "dh0")

    def loss(a):
        y, last, _ = R.gated_scan(*a[:2], "sigmoid", a[2])
        return (y * f64(dy)).sum() + (last * f64(dh)).sum()

    rng = np.random.default_rng(18)
    way = [rng.standard_normal(t.shape) for t in (dx, dg, dh0)]
    base = [f64(x), f64(g), h2]
    step = 1e-5
    diff = (loss([p + step * w for p, w in zip(base, way)]) -
            loss([p - step * w for p, w in zip(base, way)])) / (2 * step)
    got = sum((f64(p) * w).sum() for p, w in ((xs.grad, way[0]), (gs.grad, way[1])))
    got += (dh0 * way[2]).sum()
    room = sum((np.abs(w) * (b[n] + E * np.abs(v))).sum()
               for w, n, v in ((way[0], "dx", dx), (way[1], "dg", dg)))
    assert abs(got - diff) <= room + 1e-6 * abs(diff)


def test_autograd_with_one_of_the_outputs_only():
    x, g, dy, h, dh = (t.to(dev()) for t in make(2, 66, 16, F32, "log", 19))
    xs = x.clone().requires_grad_()
    _, last = S.GatedScan.apply(xs, g)
    last.sum().backward()
    a = xs.grad.clone()
    xs.grad = None
    y, _ = S.GatedScan.apply(xs, g)
    y[:, -1].sum().backward()
    assert torch.equal(a, xs.grad)
    with pytest.raises(RuntimeError):
        y, _ = S.GatedScan.apply(xs, g)
        d, = torch.autograd.grad(y.sum(), xs, create_graph=True)
        d.sum().backward()


def test_captured_training_step_replays_with_new_inputs():
    """Forward and backward in one graph, on its own stream, replayed on other data."""
    x, g, dy, h, dh = (t.to(dev()) for t in make(2, 400, 130, BF16, "log", 20))
    xs, gs, ds = x.clone(), g.clone(), dy.clone()

    def step():
        y, last, marks = S.sanatan_gated_scan_fwd(xs, gs, h0=h, want_state=True, want_marks=True)
        gr = S.sanatan_gated_scan_bwd(xs, gs, ds, marks, want_dh0=True)
        return y, last, gr["dx"], gr["dg"], gr["dh0"]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x2, g2, dy2, _, _ = (t.to(dev()) for t in make(2, 400, 130, BF16, "log", 21))
    for to, new in ((xs, x2), (gs, g2), (ds, dy2)):
        to.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_captured_autograd():
    """GatedScan's forward and backward captured as a user captures a training step."""
    x, g, dy, h, dh = (t.to(dev()) for t in make(2, 200, 72, F32, "sigmoid", 25))
    x, g, h = (t.requires_grad_() for t in (x, g, h))

    def step():
        y, last = S.GatedScan.apply(x, g, "sigmoid", h)
        return torch.autograd.grad((y * dy).sum() + (last * dh).sum(), (x, g, h))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        x.mul_(0.5)
        g.add_(0.25)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_states_updated_in_place():
    """h_out may be h0 (and dh0 dh_last): a serving state that stays where it is."""
    for B, T, D in ((1, 4000, 64), (3, 700, 100), (40, 3, 768)):
        x, g, dy, h, dh = (t.to(dev()) for t in make(B, T, D, F32, "log", T))
        y, last, marks = S.sanatan_gated_scan_fwd(x, g, h0=h, want_state=True, want_marks=True)
        state = h.clone()
        y2, _, _ = S.sanatan_gated_scan_fwd(x, g, h0=state, h_out=state)
        assert torch.equal(y, y2) and torch.equal(last, state)


def test_captured_on_joined_streams():
    """A scan that depends on two branches of a graph, and one that two depend on."""
    x, g, _, h, _ = (t.to(dev()) for t in make(2, 500, 64, F32, "sigmoid", 24))
    a, b = x.clone(), g.clone()
    S.sanatan_gated_scan_fwd(a, b, "sigmoid", h0=h)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        other.wait_stream(main)
        a.copy_(x)
        with torch.cuda.stream(other):
            b.copy_(g)
            b.mul_(2)
        main.wait_stream(other)
        y, last, _ = S.sanatan_gated_scan_fwd(a, b, "sigmoid", h0=h, want_state=True)
        other.wait_stream(main)
        with torch.cuda.stream(other):
            twice = y * 2
        step = S.sanatan_gated_scan_step(last, y[:, -1].contiguous(), h, "sigmoid")
        main.wait_stream(other)
    for scale in (1.0, -0.5):
        x.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        want, state, _ = S.sanatan_gated_scan_fwd(x, 2 * g, "sigmoid", h0=h, want_state=True)
        assert torch.equal(y, want) and torch.equal(twice, 2 * want)
        assert torch.equal(step, S.sanatan_gated_scan_step(state, want[:, -1].contiguous(), h,
                                                           "sigmoid"))


def test_first_calls_of_a_process_inside_a_capture():
    """What the library asks of the runtime once is asked while a stream captures."""
    code = """
import torch
from constant_state_recurrence_gb300 import sanatan as S
x = torch.randn(2, 300, 64, device="cuda")
g = -torch.rand(2, 300, 64, device="cuda")
state, pages = torch.randn(1, 2, 640, device="cuda"), torch.tensor([1, 0], device="cuda")
codes, scales, _ = S.state_cache_empty(2, 640)
out = torch.zeros_like(state)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, h, m = S.sanatan_gated_scan_fwd(x, g, want_state=True, want_marks=True)
    d = S.sanatan_gated_scan_bwd(x, g, y, m)
    S.sanatan_state_cache_write(state, pages, codes, scales)
    S.sanatan_state_cache_read(codes, scales, pages, out)
graph.replay()
torch.cuda.synchronize()
y2, h2, m2 = S.sanatan_gated_scan_fwd(x, g, want_state=True, want_marks=True)
d2 = S.sanatan_gated_scan_bwd(x, g, y2, m2)
assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(d["dg"], d2["dg"])
assert ((out - state).abs() <= state.abs().amax() / 250).all()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_streams_at_once():
    a = [t.to(dev()) for t in make(2, 3000, 96, F32, "log", 22)]
    b = [t.to(dev()) for t in make(3, 2500, 64, F32, "sigmoid", 23)]
    ya, _, _ = S.sanatan_gated_scan_fwd(a[0], a[1], "log", h0=a[3])
    yb, _, _ = S.sanatan_gated_scan_fwd(b[0], b[1], "sigmoid", h0=b[3])
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(one):
            y1, _, _ = S.sanatan_gated_scan_fwd(a[0], a[1], "log", h0=a[3])
        with torch.cuda.stream(two):
            y2, _, _ = S.sanatan_gated_scan_fwd(b[0], b[1], "sigmoid", h0=b[3])
    torch.cuda.synchronize()
    assert torch.equal(ya, y1) and torch.equal(yb, y2)


def test_refusals_of_the_binding():
    x = torch.zeros(2, 8, 4, device=dev())
    h = torch.zeros(2, 4, device=dev())
    for bad in (dict(g=x[:, :7]), dict(g=x.to(BF16)), dict(g=x.transpose(0, 1)),
                dict(g=x, h0=h[:1]), dict(g=x, h0=h.to(BF16)), dict(g=x, gate="relu"),
                dict(g=x, lens=torch.zeros(3, dtype=torch.int64, device=dev())),
                dict(g=x, lens=torch.zeros(2, dtype=torch.int32, device=dev())),
                dict(g=x.cpu()), dict(g=x, out=x.to(BF16)), dict(g=x, h_out=h[:, :2])):
        with pytest.raises(ValueError):
            S.sanatan_gated_scan_fwd(x, **bad)
    with pytest.raises(ValueError):
        S.sanatan_gated_scan_fwd(x[0], x[0])
    with pytest.raises(ValueError):
        S.sanatan_gated_scan_fwd(x.half(), x.half())
    with pytest.raises(S.SanatanError) as e:        # rows of 5 floats: the second is misaligned
        odd = torch.zeros(3, 1, 5, device=dev())
        S.sanatan_gated_scan_fwd(odd[1:], odd[1:])
    assert e.value.status == 1
    with pytest.raises(ValueError):
        S.sanatan_gated_scan_bwd(x, x, x, torch.zeros(2, 2, 4, device=dev()))
    with pytest.raises(ValueError):
        S.sanatan_gated_scan_step(h.to(BF16), h, h)
    with pytest.raises(ValueError):
        S.sanatan_gated_scan_step(x, x, x)
    with pytest.raises(S.SanatanError) as e:        # an output over an input
        S.sanatan_gated_scan_fwd(x, x, out=x)
    assert e.value.status == 1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D", [(1, 40, 7), (2, 70, 64), (3, 200, 771), (2, 130, 768)])
def test_autograd_with_gradients_at_any_address(B, T, D, dtype):
    """Outputs that are joined behind others get slices of one gradient back: contiguous,
    but at any element."""
    x, g, dy, h, dh = make(B, T, D, dtype, "sigmoid", 26)
    xs, gs, h0 = (t.to(dev()).requires_grad_() for t in (x, g, h))
    y, last = S.GatedScan.apply(xs, gs, "sigmoid", h0)
    where = []
    y.register_hook(lambda t: where.append(t.data_ptr() % 16))
    last.register_hook(lambda t: where.append(t.data_ptr() % 16))
    ys = torch.cat([torch.zeros(3, dtype=dtype, device=dev()), y.flatten()])
    ls = torch.cat([torch.zeros(1, device=dev()), last.flatten()])
    front = torch.ones(3, dtype=dtype)
    wy = torch.cat([front, dy.flatten()]).to(dev())
    wl = torch.cat([torch.ones(1), dh.flatten()]).to(dev())
    torch.autograd.backward([ys, ls], [wy, wl])
    assert len(where) == 2 and all(where)
    dx, dg, dh0 = R.gated_scan_backward(f64(x), f64(g), "sigmoid", f64(dy), f64(h), None, f64(dh))
    b = bounds(f64(x), f64(g), "sigmoid", f64(h), f64(dy), f64(dh))
    close(xs.grad, dx, b["dx"], dtype, "dx")
    close(gs.grad, dg, b["dg"], dtype, "dg")
    close(h0.grad, dh0, b["dh0"], F32, "dh0")


@pytest.mark.parametrize("D", [64, 70])
def test_lengths_out_of_a_longer_list(D):
    """lens[1:] of a batch's list starts at 8 bytes, not at 16."""
    x, g, dy, h, _ = (t.to(dev()) for t in make(3, 150, D, F32, "sigmoid", 27))
    lens = torch.tensor([9, 150, 31, 0], device=dev())
    assert lens[1:].data_ptr() % 16 == 8

    def both(n):
        y, last, marks = S.sanatan_gated_scan_fwd(x, g, "sigmoid", h0=h, lens=n, want_state=True,
                                                  want_marks=True)
        gr = S.sanatan_gated_scan_bwd(x, g, dy, marks, "sigmoid", lens=n, want_dh0=True)
        return y, last, gr["dx"], gr["dg"], gr["dh0"]

    assert all(torch.equal(a, b) for a, b in zip(both(lens[1:]), both(lens[1:].clone())))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,D", [(90, 771), (300, 64), (1, 5)])
def test_states_of_one_sequence_out_of_a_batch(T, D, dtype):
    """h[b:b + 1] of a batch's states (odd widths: at any float): as initial, last and step's
    state, updated where it is; the others stay as they were."""
    x, g, dy, h, dh = (t.to(dev()) for t in make(1, T, D, dtype, "log", 28))
    many = torch.randn(3 * D + 2, device=dev())
    slot, gslot = many[2:].view(3, D)[1:2], torch.cat([many[:1], dh[0]])[1:].view(1, D)
    assert slot.data_ptr() % 16 and gslot.data_ptr() % 16
    slot.copy_(h)
    kept = many.clone()
    y, last, marks = S.sanatan_gated_scan_fwd(x, g, h0=h, want_state=True, want_marks=True)
    y2, _, _ = S.sanatan_gated_scan_fwd(x, g, h0=slot, h_out=slot)
    assert torch.equal(y, y2) and torch.equal(slot, last)
    a = S.sanatan_gated_scan_bwd(x, g, dy, marks, dh_last=dh, want_dh0=True)
    b = S.sanatan_gated_scan_bwd(x, g, dy, marks, dh_last=gslot, want_dh0=True)
    assert all(torch.equal(a[n], b[n]) for n in a)
    one = S.sanatan_gated_scan_step(last, x[:, 0].contiguous(), g[:, 0].contiguous())
    two = S.sanatan_gated_scan_step(slot, x[:, 0].contiguous(), g[:, 0].contiguous())
    assert torch.equal(one, two) and torch.equal(slot, last)
    kept[2 + D:2 + 2 * D] = many[2 + D:2 + 2 * D]
    assert torch.equal(kept, many)


def decays(g, gate):
    """The decays that step, scan and backward use: of a state 1 with nothing added, and of
    a gradient 1 with nothing added."""
    g = g.view(1, -1)
    zero, one = torch.zeros_like(g), torch.ones_like(g)
    h = one.clone()
    S.sanatan_gated_scan_step(h, zero, g, gate)
    g3, zero3 = g[:, None], zero[:, None]
    y, _, marks = S.sanatan_gated_scan_fwd(zero3, g3, gate, h0=one, want_marks=True)
    d = S.sanatan_gated_scan_bwd(zero3, g3, zero3, marks, gate, dh_last=one, want_dh0=True)
    assert torch.equal(h, y[:, 0]) and torch.equal(h, d["dh0"])
    return f64(h)[0]


@pytest.mark.parametrize("odd", [0, 1])
def test_decays_next_to_one(odd):
    """Steps E = 2^-24 of the decay itself.  Log gate, |g| < 1/16: the last of five terms
    rounds by E / 2, the ones within by |g| E / 2 and |g|^2 E / 4 and less (1.07 E / 2 at
    1/16), and the sixth, left out, is g^5 / 120 <= 0.134 E: 0.67 E, and on average (the
    roundings come out even; the sixth term averages to 0.022 E, the inner ones to at most
    0.035 E) less than 0.08 E.  Sigmoid, g > 2.8: e = exp(-g) is within (4 + 2 g) E of its
    value (power of two 4 E, its argument 2 g E), which moves the decay 1 / (1 + e) by at
    most 1 - a times that; rounding it once adds E / 2, the reciprocal's error squared
    nothing to speak of (4 (1 - a) E are more than that)."""
    n = (1 << 16) + odd
    gen = torch.Generator().manual_seed(29 + odd)
    g = -torch.rand(n, generator=gen) / 16
    off = decays(g.to(dev()), "log") - np.exp(f64(g))
    assert np.abs(off).max() <= 0.67 * E
    assert abs(off.mean()) <= 0.08 * E
    g = 2.8 + 9 * torch.rand(n, generator=gen)
    keep = 1 / (1 + np.exp(f64(g)))
    off = decays(g.to(dev()), "sigmoid") - (1 - keep)
    assert (np.abs(off) <= (0.5 + keep * (8 + 2 * f64(g))) * E).all()


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("D", [64, 61])
def test_constant_gates_next_to_one(gate, D):
    """Gates that do not change from token to token, whose decays' errors do not average out,
    over 32768 tokens of input 1.  A token adds its decay's error (see above), one product
    of decays (a tree of products has fewer than a token each: E / 2 of a product above 3/4) and
    a sixteenth of an addition to the state: together under 3 E / 4; and a scan in pieces
    40 E of the state on its way."""
    T = 32768
    if gate == "log":
        g = -torch.logspace(-4, -3, D)
        k = np.full(D, 0.67 * E)
        a, u = np.exp(f64(g)), np.ones(D)
    else:
        g = torch.linspace(7, 10, D)
        u = 1 / (1 + np.exp(f64(g)))
        k = (0.5 + u * (8 + 2 * f64(g))) * E
        a = 1 - u
    x = torch.ones(1, T, D, device=dev())
    y, last, _ = S.sanatan_gated_scan_fwd(x, g.to(dev()).expand(1, T, D).contiguous(), gate,
                                          want_state=True)
    n = np.arange(1, T + 1)[:, None]
    ref = u * -np.expm1(n * np.log(a)) / (1 - a)                   # u (1 - a^n) / (1 - a)
    err = np.zeros(D)
    room = np.zeros((T, D))
    ku = (8 + 2 * np.abs(f64(g))) * E * (gate == "sigmoid")
    for t in range(T):
        before = ref[t - 1] if t else np.zeros(D)
        err = a * err + (k + 0.75 * E) * before + ku * u
        room[t] = err + 40 * E * ref[t]
    close(y[0], ref, room, F32, "y")
    close(last[0], ref[-1], room[-1], F32, "last")


@pytest.mark.parametrize("dtype,D", [(BF16, 22000), (BF16, 22001)])
def test_offsets_beyond_32_bits_backward_and_odd_rows(dtype, D):
    """More than 2^31 elements, rows of 16 bytes and odd ones: the last sequence's outputs
    and gradients are where they should be.  a = 1: sums forward and backward in time."""
    B, T = 3, 32768
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.zeros(B, T, D, dtype=dtype, device=dev())
    g = torch.zeros_like(x)
    dy = torch.zeros_like(x)
    c = torch.arange(D, device=dev()).remainder(251).to(dtype)
    x[2, -130], x[2, -2] = 1.0, c
    dy[2, -1], dy[2, 5] = c, 2.0
    y, last, marks = S.sanatan_gated_scan_fwd(x, g, want_state=True, want_marks=True)
    assert torch.equal(last[2], c.float() + 1) and not last[:2].any()
    assert torch.equal(y[2, -1], (c.float() + 1).to(dtype)) and (y[2, -130:-2] == 1).all()
    assert not y[2, :-130].any() and not y[:2].any()
    d = S.sanatan_gated_scan_bwd(x, g, dy, marks, want_dh0=True)
    dx, dg = d["dx"], d["dg"]
    assert torch.equal(dx[2, 6], c) and torch.equal(dx[2, -1], c)
    assert torch.equal(dx[2, 5], (c.float() + 2).to(dtype)) and torch.equal(dx[2, 0], dx[2, 5])
    assert not dx[:2].any() and not dg[:2].any() and not dg[2, :-129].any()
    assert (dg[2, -129:-1] == c).all()                              # dh a h, h = 1 before
    assert torch.equal(dg[2, -1], (c.float() * (c.float() + 1)).to(dtype))
    assert torch.equal(d["dh0"][2], c.float() + 2) and not d["dh0"][:2].any()
    S.device_status()


@pytest.mark.parametrize("D", [64, 66])
def test_gates_above_zero_grow(D):
    """The log gate above 0, up to products of all decays next to the largest float32: what
    the formula gives; zeros stay zeros."""
    T = 300
    x, g, dy, h, dh = make(2, T, D, F32, "log", 30)
    g = torch.where(torch.arange(D) % 2 == 0, g + 0.5, torch.tensor(80.0 / T)).contiguous()
    d = lambda t: t.to(dev())  # noqa: E731
    y, last, marks = S.sanatan_gated_scan_fwd(d(x), d(g), h0=d(h), want_state=True,
                                              want_marks=True)
    ref, last_ref, _ = R.gated_scan(f64(x), f64(g), "log", f64(h))
    b = bounds(f64(x), f64(g), "log", f64(h))
    close(y, ref, b["y"], F32, "y")
    close(last, last_ref, b["last"], F32, "last")
    zero = torch.zeros_like(d(x))
    y, last, _ = S.sanatan_gated_scan_fwd(zero, d(g), want_state=True)
    assert not y.any() and not last.any()
