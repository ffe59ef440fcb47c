"""The short causal convolution on the GPU (forward, backward, single-token step, autograd)
against the float64 definitions.

Tolerances, element by element, in steps e = 2^-24 of float32: c has K + 1 roundings, Ec =
(K + 2) e sum|w x|; c / (1 + exp(-c)) has a slope below 1.1 and is formed within (10 + 2 |c|)
e of its value (exponential 2 ulp, its argument's rounding |c| e, sum, division 2 ulp).
The slope itself changes by at most 0.5 for one of c and is formed within (24 + 4 |c|) e of
its two terms, sg and c sg (1 - sg).  Sums over tokens have at most 160 additions on the way
(32 tokens a run, runs of a thread, eight of a block, blocks), sums over taps K.  An output in
bf16 is off by half a step more, 2^-8 of its value (float32: 2^-24); 1e-36 stands for underflow."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as R
from constant_state_recurrence_gb300 import sanatan as S
from gpu_util import dev, f64
from test_gpu_layer_norm import BF16, E, F32, close

pytestmark = pytest.mark.gpu


def make(B, T, D, K, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, dy = n(B, T, D).to(dtype), n(B, T, D).to(dtype)
    return x, n(D, K), 0.3 * n(D), dy, n(B, K - 1, D), n(B, K - 1, D)


def bounds(x, w, bias, silu, s0, lens, dy=None, ds=None):
    """Bounds of y, dx, dw, dbias and ds0, from the definitions of the magnitudes."""
    K = w.shape[1]
    m = np.abs
    _, _, c = R.causal_conv(x, w, bias, False, s0, lens)
    _, _, mag = R.causal_conv(m(x), m(w), None if bias is None else m(bias), False,
                              None if s0 is None else m(s0), lens)
    Ec = (K + 2) * E * mag
    sg = R.sigmoid(c)
    out = dict(y=1.1 * Ec + (10 + 2 * m(c)) * E * m(c * sg) if silu else Ec)
    if dy is None:
        return out
    slope = R.silu_slope(c) if silu else np.ones_like(c)
    Ed = m(dy) * (0.5 * Ec + (24 + 4 * m(c)) * E * (sg + m(c) * sg * (1 - sg))) if silu else 0 * dy
    # dx, dw and dbias of |dc| with |w| and |x|, and of its error
    dc, z = m(dy * slope), None if s0 is None else m(s0)
    top = R.causal_conv_backward(m(x), m(w), dc, None, False, z, lens, None if ds is None else m(ds))
    err = R.causal_conv_backward(m(x), m(w), Ed, None, False, z, lens, None)
    steps = ((K + 3) * E, 160 * E, 160 * E, (K + 3) * E)
    for name, t, e, k in zip(("dx", "dw", "dbias", "ds0"), top, err, steps):
        out[name] = e + k * (t + e)
    return out


def check(B, T, D, K, dtype, silu=True, s0=True, lens=None, seed=0, biased=True, ld=None,
          place=lambda t: t.to(dev())):
    x, w, bias, dy, s, ds = make(B, T, D, K, dtype, seed)
    d = lambda t: None if t is None else place(t)  # noqa: E731
    s, ds = (s, ds) if s0 else (None, None)
    bias = bias if biased else None
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int64).to(dev())
    xd = d(x)
    if ld:
        wide = torch.full((B, T, ld), float("nan"), dtype=dtype, device=dev())
        wide[..., ld - D:] = xd
        xd = wide[..., ld - D:]
    act = "silu" if silu else None
    y, last = S.sanatan_causal_conv_fwd(xd, d(w), d(bias), act, s0=d(s), lens=ln, want_state=True)
    g = S.sanatan_causal_conv_bwd(xd, d(w), d(dy), d(bias), act, s0=d(s), lens=ln, ds_last=d(ds),
                                  want_ds0=True)
    torch.cuda.synchronize()
    n = lambda t: None if t is None else f64(t)  # noqa: E731
    cut = None if lens is None else R.lengths(lens, B, T)
    yr, lr, _ = R.causal_conv(n(x), n(w), n(bias), silu, n(s), cut)
    ref = R.causal_conv_backward(n(x), n(w), n(dy), n(bias), silu, n(s), cut, n(ds))
    bd = bounds(n(x), n(w), n(bias), silu, n(s), cut, n(dy), n(ds))
    there = np.ones((B, T, 1)) if cut is None else \
        (np.arange(T)[None] < np.asarray(cut)[:, None])[..., None]
    close(y, yr, bd["y"] * there, dtype, "y")
    assert np.array_equal(f64(last), lr)
    for name, r, ty in zip(("dx", "dw", "dbias", "ds0"), ref, (dtype, F32, F32, F32)):
        close(g[name], r, bd[name] * (there if name == "dx" else 1), ty, name)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D,K", [
    (1, 1, 1, 1), (1, 1, 4, 4), (2, 2, 3, 4), (1, 3, 8, 8), (3, 5, 7, 3), (2, 16, 64, 4),
    (1, 17, 12, 2), (2, 31, 33, 5), (1, 32, 128, 4), (2, 33, 130, 4), (3, 66, 20, 7), (1, 200, 5, 6),
    (5, 100, 260, 4), (1, 300, 36, 3), (70, 3, 8, 4)])
def test_against_the_definition(B, T, D, K, dtype):
    check(B, T, D, K, dtype, silu=(T + K) % 3 != 0, s0=T % 2 == 1, seed=T + D, biased=D % 5 != 0)


@pytest.mark.parametrize("D", [64, 31])
@pytest.mark.parametrize("K", [1, 2, 4, 8])
def test_lengths_and_states(K, D):
    """From no token to all, shorter than the taps, values outside [0, T]."""
    check(7, 40, D, K, F32, lens=[0, 1, 2, 40, 33, -5, 1000], seed=K)
    check(3, 2, D, K, BF16, lens=[2, 0, 1], seed=K + 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,ld", [(64, 128), (64, 65), (33, 70), (8, 16)])
def test_a_half_of_a_wider_projection(D, ld, dtype):
    check(2, 37, D, 4, dtype, ld=ld, seed=ld)


def test_parts_of_larger_tensors():
    def place(t):
        big = torch.zeros(t.numel() + 1, dtype=t.dtype, device=dev())
        big[1:].copy_(t.flatten())
        return big[1:].view(t.shape)
    check(2, 37, 64, 4, BF16, lens=[37, 20], place=place)
    check(2, 37, 64, 3, F32, place=place)


def test_no_tokens_and_no_sequences():
    x, w, bias, dy, s, ds = (t.to(dev()) for t in make(3, 0, 12, 4, F32, 1))
    y, last = S.sanatan_causal_conv_fwd(x, w, bias, s0=s, want_state=True)
    assert y.shape == (3, 0, 12) and torch.equal(last, s)
    g = S.sanatan_causal_conv_bwd(x, w, dy, bias, s0=s, ds_last=ds, want_ds0=True)
    assert torch.equal(g["ds0"], ds) and not g["dw"].any() and not g["dbias"].any()
    x, w, bias, dy, s, ds = (t.to(dev()) for t in make(0, 5, 12, 4, F32, 1))
    g = S.sanatan_causal_conv_bwd(x, w, dy, bias)
    assert not g["dw"].any() and not g["dbias"].any()


@pytest.mark.parametrize("dtype,D", [(F32, 100), (BF16, 64), (BF16, 7)])
@pytest.mark.parametrize("K", [1, 4, 6])
def test_pieces_and_single_tokens_are_the_whole(K, D, dtype):
    """The same sums in the same order: equal to the bit."""
    x, w, bias, _, s, _ = (t.to(dev()) for t in make(3, 50, D, K, dtype, 2))
    y, last = S.sanatan_causal_conv_fwd(x, w, bias, s0=s, want_state=True)
    a, state = S.sanatan_causal_conv_fwd(x[:, :21].contiguous(), w, bias, s0=s, want_state=True)
    b, state = S.sanatan_causal_conv_fwd(x[:, 21:49].contiguous(), w, bias, s0=state,
                                         want_state=True)
    c = S.sanatan_causal_conv_step(state, x[:, 49], w, bias)
    assert torch.equal(torch.cat([a, b, c.unsqueeze(1)], 1), y) and torch.equal(state, last)


def test_what_is_behind_a_sequence_is_not_read():
    x, w, bias, dy, s, ds = (t.to(dev()) for t in make(2, 40, 36, 4, F32, 3))
    lens = torch.tensor([22, 0], device=dev())

    def all_of(x, dy):
        y, last = S.sanatan_causal_conv_fwd(x, w, bias, s0=s, lens=lens, want_state=True)
        g = S.sanatan_causal_conv_bwd(x, w, dy, bias, s0=s, lens=lens, ds_last=ds, want_ds0=True)
        return [y, last] + [g[k] for k in ("dx", "dw", "dbias", "ds0")]

    want = all_of(x, dy)
    for t in (x, dy):
        t[0, 22:] = float("nan")
        t[1] = float("inf")
    assert all(torch.equal(p, q) for p, q in zip(want, all_of(x, dy)))


def test_a_value_that_is_not_finite_reaches_its_window_only():
    for K, D in ((3, 64), (7, 10)):
        x, w, bias, _, _, _ = (t.to(dev()) for t in make(1, 60, D, K, F32, 4))
        y, _ = S.sanatan_causal_conv_fwd(x, w, bias, None)
        x[0, 20, 5] = float("inf")
        bad, _ = S.sanatan_causal_conv_fwd(x, w, bias, None)
        hit = torch.zeros(1, 60, D, dtype=torch.bool, device=dev())
        hit[0, 20:20 + K, 5] = True
        assert torch.equal(y[~hit], bad[~hit]) and not bad[hit].isfinite().any()


def test_autograd_with_a_half_of_a_projection():
    x, w, bias, dy, s, ds = (t.to(dev()) for t in make(2, 30, 40, 4, F32, 5))
    wide = torch.randn(2, 30, 80, device=dev()).requires_grad_()
    leaves = [t.clone().requires_grad_() for t in (w, bias, s)]
    y, last = S.CausalConv.apply(wide[..., 40:], leaves[0], leaves[1], "silu", leaves[2])
    ((y * dy).sum() + (last * ds).sum()).backward()
    x64 = f64(wide[..., 40:])
    ref = R.causal_conv_backward(x64, f64(w), f64(dy), f64(bias), True, f64(s), None, f64(ds))
    bd = bounds(x64, f64(w), f64(bias), True, f64(s), None, f64(dy), f64(ds))
    assert not wide.grad[..., :40].any()
    for got, r, name in zip((wide.grad[..., 40:], leaves[0].grad, leaves[1].grad, leaves[2].grad),
                            ref, ("dx", "dw", "dbias", "ds0")):
        close(got, r, bd[name], F32, name)
    _, last = S.CausalConv.apply(x.requires_grad_(), w, bias)
    last.sum().backward()
    want = torch.zeros_like(x)
    want[:, -3:] = 1
    assert torch.equal(x.grad, want)


def test_captured_step_and_training_step():
    x, w, bias, dy, s, ds = (t.to(dev()) for t in make(4, 90, 72, 4, BF16, 6))
    state = s.clone()

    def step():
        y, last = S.sanatan_causal_conv_fwd(x, w, bias, s0=s, want_state=True)
        g = S.sanatan_causal_conv_bwd(x, w, dy, bias, s0=s)
        return y, last, g["dx"], g["dw"], g["dbias"]

    step(), S.sanatan_causal_conv_step(state, x[:, 0], w, bias)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
        one = S.sanatan_causal_conv_step(state, x[:, 0], w, bias)
    x.mul_(0.5)
    state.copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, step()))
    again = s.clone()
    assert torch.equal(one, S.sanatan_causal_conv_step(again, x[:, 0], w, bias))
    assert torch.equal(state, again)


def test_refusals():
    x, w, bias, dy, s, ds = (t.to(dev()) for t in make(2, 9, 16, 4, F32, 7))
    for bad in (lambda: S.sanatan_causal_conv_fwd(x, torch.ones(16, 9, device=dev())),
                lambda: S.sanatan_causal_conv_fwd(x, w, activation="relu"),
                lambda: S.sanatan_causal_conv_fwd(x, w[:8], bias),
                lambda: S.sanatan_causal_conv_fwd(x.transpose(0, 1), w, bias),
                lambda: S.sanatan_causal_conv_fwd(x[:, :1].expand(2, 9, 16), w, bias),
                lambda: S.sanatan_causal_conv_fwd(x[..., ::2], w[::2].contiguous()),
                lambda: S.sanatan_causal_conv_fwd(x.double(), w),
                lambda: S.sanatan_causal_conv_fwd(x, w, s0=s[:, :2].contiguous()),
                lambda: S.sanatan_causal_conv_fwd(x, w, lens=torch.ones(2, device=dev())),
                lambda: S.sanatan_causal_conv_step(s.bfloat16(), x[:, 0], w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: S.sanatan_causal_conv_fwd(x, w, out=x),
                lambda: S.sanatan_causal_conv_fwd(x, w, s0=s, s_out=s)):
        with pytest.raises(S.SanatanError):
            bad()
