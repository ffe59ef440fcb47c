"""The layer norm on the GPU (forward, backward, autograd) against the float64 definitions.

Tolerances, element by element, in steps e = 2^-24 of float32.  A sum of D values over
threads, lanes and warps has at most k = 48 + D / 512 additions on the way of a value,
so a mean is off by (k + 2) e times the mean magnitude, and the variance, formed from the
differences, by twice that times the mean difference and (k + 4) e of itself; division and
root add 3 e.  n = (s - mean) rstd and what is formed from it follow by the product
rule.  Sums over rows have at most 100 + rows / 100 additions on the way.  An output in bf16
is off by half a step more, 2^-8 of its value (float32: 2^-24); 1e-36 stands for underflow.
The residual sum is the exact sum rounded once, and equal."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as R
from constant_state_recurrence_gb300 import sanatan as S
from gpu_util import dev, f64

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def make(rows, D, dtype, seed, mean=0.3):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, r, dy, ds = n(rows, D) + mean, n(rows, D), n(rows, D), n(rows, D)
    return [t.to(dtype) for t in (x, r, dy, ds)] + [1 + 0.3 * n(D), 0.2 * n(D)]


def close(got, ref, bound, dtype, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    room = bound * (1 + 1e-3) + HALF[dtype] * (np.abs(ref) + bound) + 1e-36
    off = np.abs(got - ref) - room
    assert np.isfinite(got).all(), what
    assert off.max(initial=-1.0) <= 0, (what, np.unravel_index(off.argmax(), off.shape), off.max())


def bounds(s, w, b, dy=None, ds=None, eps=EPS):
    rows, D = s.shape
    k = 48 + D / 512
    y, mean, rstd = R.layer_norm(s, w, b, eps)
    d = s - mean[:, None]
    em = (k + 2) * E * np.abs(s).mean(-1)
    var = (d ** 2).mean(-1)
    ev = 2 * em * np.abs(d).mean(-1) + em ** 2 + (k + 4) * E * var
    rr = (0.5 * ev / (var + eps) + 4 * E)[:, None]              # relative, of rstd
    hat, em, r1 = d * rstd[:, None], em[:, None], rstd[:, None]
    eh = np.abs(hat) * (rr + 3 * E) + em * r1 * (1 + rr)
    out = dict(y=np.abs(w) * (eh + 2 * E * np.abs(hat)) + E * np.abs(y))
    if dy is None:
        return out
    m = lambda v: v.mean(-1, keepdims=True)  # noqa: E731
    g = dy * w
    e1 = (k + 3) * E * m(np.abs(g))
    e2 = m(np.abs(g) * eh) + (k + 5) * E * m(np.abs(g * hat))
    c1, c2 = m(g), m(g * hat)
    t = g - c1 - hat * c2
    et = E * np.abs(g) + e1 + np.abs(hat) * e2 + np.abs(c2) * eh + eh * e2 \
        + 4 * E * (np.abs(g) + np.abs(c1) + np.abs(hat * c2))
    out["dx"] = r1 * (et + (rr + 3 * E) * (np.abs(t) + et)) \
        + (0 if ds is None else 2 * E * np.abs(ds))
    n = 100 + rows / 100
    out["dw"] = (np.abs(dy) * eh).sum(0) + n * E * np.abs(dy * hat).sum(0)
    out["db"] = n * E * np.abs(dy).sum(0)
    return out


def check(rows, D, dtype, residual, seed=0, mean=0.3, place=lambda t: t.to(dev())):
    x, r, dy, ds, w, b = make(rows, D, dtype, seed, mean)
    d = place
    y, s, stats = S.sanatan_layer_norm_fwd(d(x), d(w), d(b), d(r) if residual else None, EPS,
                                           want_stats=True)
    gr = S.sanatan_layer_norm_bwd(d(x) if s is None else s, d(w), d(dy), stats,
                                  ds=d(ds) if residual else None)
    torch.cuda.synchronize()
    if residual:
        total = (x.double() + r.double()).to(dtype)
        assert torch.equal(s.cpu(), total)
    else:
        total = x
    s64, w64, b64, dy64 = f64(total), f64(w), f64(b), f64(dy)
    ds64 = f64(ds) if residual else None
    bd = bounds(s64, w64, b64, dy64, ds64)
    close(y, R.layer_norm(s64, w64, b64, EPS)[0], bd["y"], dtype, "y")
    dx, dw, db = R.layer_norm_backward(s64, w64, dy64, ds64, EPS)
    close(gr["dx"], dx, bd["dx"], dtype, "dx")
    close(gr["dweight"], dw, bd["dw"], F32, "dweight")
    close(gr["dbias"], db, bd["db"], F32, "dbias")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,D", [
    (1, 1), (1, 8), (2, 3), (5, 33), (3, 64), (4, 255), (9, 256), (2, 257), (1, 768), (77, 768),
    (6, 771), (5, 1000), (3, 1024), (4, 1025), (2, 1536), (7, 2048), (3, 4096), (2, 4104),
    (2, 8192), (3, 8193), (2, 8200), (2, 20000), (3000, 24), (2500, 96), (1300, 260)])
def test_against_the_definition(rows, D, dtype):
    check(rows, D, dtype, residual=(rows + D) % 2 == 0, seed=rows + D)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 768, 2048, 9000])
def test_parts_of_larger_tensors(D, dtype):
    """Addresses at any element (and weights, too): the same formulas."""
    def place(t):
        big = torch.zeros(t.numel() + 3, dtype=t.dtype, device=dev())
        big[3:].copy_(t.flatten())
        return big[3:].view(t.shape)
    check(5, D, dtype, residual=True, seed=D, place=place)


@pytest.mark.parametrize("D", [768, 5000])
def test_a_mean_far_from_zero(D):
    check(6, D, F32, residual=False, seed=3, mean=3e4)


def test_without_weight_and_bias():
    x, _, dy, _, _, _ = make(9, 200, F32, 4)
    y, s, stats = S.sanatan_layer_norm_fwd(x.to(dev()), want_stats=True)
    assert s is None
    d = S.sanatan_layer_norm_bwd(x.to(dev()), None, dy.to(dev()), stats, want_dweight=False,
                                 want_dbias=False)
    one = np.ones(200)
    bd = bounds(f64(x), one, 0 * one, f64(dy))
    close(y, R.layer_norm(f64(x))[0], bd["y"], F32, "y")
    close(d["dx"], R.layer_norm_backward(f64(x), None, f64(dy))[0], bd["dx"], F32, "dx")
    assert d["dweight"] is None and d["dbias"] is None
    w = torch.ones(200, device=dev())
    only = S.sanatan_layer_norm_bwd(x.to(dev()), w, dy.to(dev()), stats, want_dbias=False)
    both = S.sanatan_layer_norm_bwd(x.to(dev()), w, dy.to(dev()), stats)
    assert torch.equal(only["dweight"], both["dweight"]) and torch.equal(only["dx"], both["dx"])


def test_no_rows():
    x = torch.zeros(0, 40, device=dev())
    y, s, stats = S.sanatan_layer_norm_fwd(x, residual=x, want_stats=True)
    assert y.shape == s.shape == (0, 40) and stats.shape == (0, 2)
    d = S.sanatan_layer_norm_bwd(x, torch.ones(40, device=dev()), x, stats)
    assert not d["dweight"].any() and not d["dbias"].any() and d["dx"].shape == (0, 40)


@pytest.mark.parametrize("D", [768, 771, 3000, 9001])
def test_the_stream_in_place_and_the_same_bits(D):
    x, r, dy, ds, w, b = (t.to(dev()) for t in make(300, D, BF16, 5))
    y, s, stats = S.sanatan_layer_norm_fwd(x, w, b, r, want_stats=True)
    a = S.sanatan_layer_norm_bwd(s, w, dy, stats, ds)
    stream = r.clone()
    y2, s2, stats2 = S.sanatan_layer_norm_fwd(x, w, b, stream, sum_out=stream, want_stats=True)
    c = S.sanatan_layer_norm_bwd(s, w, dy, stats2, ds)
    assert s2 is stream
    for p, q in [(y, y2), (s, s2), (stats, stats2)] + [(a[k], c[k]) for k in a]:
        assert torch.equal(p, q)


def test_a_row_that_is_not_finite_stays_alone():
    for D in (64, 2000, 9000):
        x, r, dy, ds, w, b = (t.to(dev()) for t in make(9, D, F32, 6))
        y, s, stats = S.sanatan_layer_norm_fwd(x, w, b, r, want_stats=True)
        d = S.sanatan_layer_norm_bwd(s, w, dy, stats, ds)
        x[4, 1] = float("nan")
        y2, s2, stats2 = S.sanatan_layer_norm_fwd(x, w, b, r, want_stats=True)
        d2 = S.sanatan_layer_norm_bwd(s2, w, dy, stats2, ds)
        rest = [i for i in range(9) if i != 4]
        assert torch.equal(y[rest], y2[rest]) and torch.equal(d["dx"][rest], d2["dx"][rest])
        assert y2[4].isnan().all()


def test_autograd_of_a_residual_branch():
    x, r, dy, ds, w, b = (t.to(dev()) for t in make(21, 96, F32, 7))
    leaves = [t.clone().requires_grad_() for t in (x, w, b, r)]
    y, s = S.LayerNorm.apply(*leaves)
    ((y * dy).sum() + (s * ds).sum()).backward()
    total = f64(s)
    dx, dw, db = R.layer_norm_backward(total, f64(w), f64(dy), f64(ds), EPS)
    bd = bounds(total, f64(w), f64(b), f64(dy), f64(ds))
    for leaf, ref, n in zip(leaves, (dx, dw, db, dx), ("dx", "dw", "db", "dx")):
        close(leaf.grad, ref, bd[n], F32, n)
    leaves = [t.clone().requires_grad_() for t in (x, w)]
    S.LayerNorm.apply(*leaves).sum().backward()      # a gradient that is one number, spread out
    ref = R.layer_norm_backward(f64(x), f64(w), np.ones(x.shape))[0]
    close(leaves[0].grad, ref, bounds(f64(x), f64(w), 0, np.ones(x.shape))["dx"], F32, "dx")


def test_captured_and_on_another_stream():
    x, r, dy, ds, w, b = (t.to(dev()) for t in make(400, 768, BF16, 8))

    def step():
        y, s, stats = S.sanatan_layer_norm_fwd(x, w, b, r, want_stats=True)
        d = S.sanatan_layer_norm_bwd(s, w, dy, stats, ds)
        return y, s, d["dx"], d["dweight"], d["dbias"]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(there, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, step()))


def test_refusals():
    x, r, dy, ds, w, b = (t.to(dev()) for t in make(4, 16, F32, 9))
    y, s, stats = S.sanatan_layer_norm_fwd(x, w, b, r, want_stats=True)
    for bad in (lambda: S.sanatan_layer_norm_fwd(x.half(), w, b),
                lambda: S.sanatan_layer_norm_fwd(x.t(), w, b),
                lambda: S.sanatan_layer_norm_fwd(x, w[:8], b),
                lambda: S.sanatan_layer_norm_fwd(x, w.bfloat16(), b),
                lambda: S.sanatan_layer_norm_fwd(x, w, b, r.bfloat16()),
                lambda: S.sanatan_layer_norm_fwd(x, w, b, sum_out=s),
                lambda: S.sanatan_layer_norm_fwd(x.cpu(), w, b),
                lambda: S.sanatan_layer_norm_bwd(s, w, dy[:2], stats),
                lambda: S.sanatan_layer_norm_bwd(s, w, dy, stats[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(S.SanatanError):
        S.sanatan_layer_norm_fwd(x, w, b, out=x)
    with pytest.raises(S.SanatanError):
        S.sanatan_layer_norm_bwd(s, w, dy, stats,
                                 workspace=torch.empty(4, dtype=torch.uint8, device=dev()))
