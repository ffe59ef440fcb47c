"""Pins of the float64 definitions in oracle/layer_oracle.py: closed forms, brute force
and finite differences."""
import numpy as np
import pytest

import oracle.layer_oracle as R


def rng(seed):
    return np.random.default_rng(seed)


def by_differences(loss, values, grads, seed, step=1e-6, bar=2e-7):
    """A gradient along a random direction against the loss on both sides."""
    r = rng(seed)
    way = [r.standard_normal(v.shape) for v in values]
    both = [loss([v + s * step * w for v, w in zip(values, way)]) for s in (1, -1)]
    want = sum((g * w).sum() for g, w in zip(grads, way))
    assert abs((both[0] - both[1]) / (2 * step) - want) <= bar * (1 + abs(want))


def test_norm_of_two_values_and_its_invariances():
    s = np.array([[1.0, 3.0]])
    y, mean, rstd = R.layer_norm(s, eps=0.0)
    assert np.array_equal(y, [[-1.0, 1.0]]) and mean[0] == 2.0 and rstd[0] == 1.0
    s = rng(0).standard_normal((3, 17))
    y = R.layer_norm(s, eps=0.0)[0]
    assert np.abs(y - R.layer_norm(5 * s + 7, eps=0.0)[0]).max() <= 1e-12
    assert np.abs(y.mean(-1)).max() <= 1e-14 and np.abs((y ** 2).mean(-1) - 1).max() <= 1e-14


def test_norm_gradients_by_differences():
    r = rng(1)
    s, dy, ds = (r.standard_normal((4, 9)) for _ in range(3))
    w, b = r.standard_normal(9), r.standard_normal(9)
    grads = R.layer_norm_backward(s, w, dy, ds, eps=1e-2)
    by_differences(lambda v: (R.layer_norm(*v, eps=1e-2)[0] * dy).sum() + (v[0] * ds).sum(),
                   [s, w, b], grads, 2)


@pytest.mark.parametrize("K", [1, 2, 4, 8])
def test_convolution_against_numpy_and_in_pieces(K):
    r = rng(K)
    x, w, bias = r.standard_normal((2, 11, 3)), r.standard_normal((3, K)), r.standard_normal(3)
    y, last, _ = R.causal_conv(x, w, bias, silu=False)
    for d in range(3):
        full = np.convolve(x[0, :, d], w[d, ::-1])[:11]
        assert np.abs(y[0, :, d] - full - bias[d]).max() <= 1e-12
    a, s, _ = R.causal_conv(x[:, :2], w, bias)
    b, s, _ = R.causal_conv(x[:, 2:], w, bias, s0=s)
    y, last, c = R.causal_conv(x, w, bias)
    assert np.abs(np.concatenate([a, b], 1) - y).max() <= 1e-12 and np.array_equal(s, last)
    assert np.abs(y - c / (1 + np.exp(-c))).max() <= 1e-14
    y2, s2, _ = R.causal_conv(x, w, bias, lens=[5, 0])
    assert np.array_equal(y2[0, :5], y[0, :5]) and not y2[0, 5:].any() and not y2[1].any()
    assert not s2[1].any()


@pytest.mark.parametrize("K,silu", [(1, True), (3, False), (4, True)])
def test_convolution_gradients_by_differences(K, silu):
    r = rng(10 + K)
    x, s0 = r.standard_normal((2, 6, 3)), r.standard_normal((2, K - 1, 3))
    w, bias = r.standard_normal((3, K)), r.standard_normal(3)
    dy, ds = r.standard_normal(x.shape), r.standard_normal(s0.shape)
    lens = [6, 2]
    grads = R.causal_conv_backward(x, w, dy, bias, silu, s0, lens, ds)

    def loss(v):
        y, last, _ = R.causal_conv(v[0], v[1], v[2], silu, v[3], lens)
        return (y * dy).sum() + (last * ds).sum()

    by_differences(loss, [x, w, bias, s0], grads, 3)
    assert not grads[0][1, 2:].any()


def _inputs(b, T, D, N, seed):
    r = rng(seed)
    u, dt, z = (r.standard_normal((b, T, D)) for _ in range(3))
    return dict(u=u, dt=dt, A=-np.exp(r.standard_normal((D, N))), B=r.standard_normal((b, T, N)),
                C=r.standard_normal((b, T, N)), D=r.standard_normal(D), z=z,
                dt_bias=r.standard_normal(D), h0=r.standard_normal((b, D, N)))


def test_scan_is_the_sum_of_decayed_inputs():
    x = _inputs(1, 7, 2, 3, 20)
    y, last, _ = R.selective_scan(**x)
    delta = np.log(1 + np.exp(x["dt"] + x["dt_bias"]))[0]
    for t in range(7):
        h = np.exp(delta[:t + 1].sum(0)[:, None] * x["A"]) * x["h0"][0]
        for j in range(t + 1):
            h = h + np.exp(delta[j + 1:t + 1].sum(0)[:, None] * x["A"]) \
                * (delta[j] * x["u"][0, j])[:, None] * x["B"][0, j]
        want = (h * x["C"][0, t]).sum(-1) + x["D"] * x["u"][0, t]
        want = want * x["z"][0, t] / (1 + np.exp(-x["z"][0, t]))
        assert np.abs(y[0, t] - want).max() <= 1e-12
    assert np.abs(last[0] - h).max() <= 1e-12


def test_scan_in_pieces_with_lengths():
    x = _inputs(2, 9, 3, 2, 21)
    y, last, _ = R.selective_scan(**x)
    cut = {k: v[:, :4] if k in ("u", "dt", "B", "C", "z") else v for k, v in x.items()}
    rest = {k: v[:, 4:] if k in ("u", "dt", "B", "C", "z") else v for k, v in x.items()}
    a, h, _ = R.selective_scan(**cut)
    b, h, _ = R.selective_scan(**{**rest, "h0": h})
    assert np.abs(np.concatenate([a, b], 1) - y).max() <= 1e-12 and np.abs(h - last).max() <= 1e-12
    y2, h2, _ = R.selective_scan(**x, lens=[4, 0])
    assert np.array_equal(y2[0, :4], y[0, :4]) and not y2[0, 4:].any() and not y2[1].any()
    assert np.array_equal(h2[1], x["h0"][1])


@pytest.mark.parametrize("soft,gated", [(True, True), (False, True), (True, False)])
def test_scan_gradients_by_differences(soft, gated):
    x = _inputs(2, 5, 3, 2, 22)
    if not gated:
        x["z"] = None
    if not soft:
        x["dt"], x["dt_bias"] = np.abs(x["dt"]), np.abs(x["dt_bias"])
    r = rng(23)
    dy, dh, lens = r.standard_normal((2, 5, 3)), r.standard_normal((2, 3, 2)), [5, 3]
    names = [n for n in x if x[n] is not None]
    grads = R.selective_scan_backward(x["u"], x["dt"], x["A"], x["B"], x["C"], dy, x["D"], x["z"],
                                      x["dt_bias"], soft, x["h0"], lens, dh)

    def loss(v):
        y, h, _ = R.selective_scan(**{**x, **dict(zip(names, v))}, soft=soft, lens=lens)
        return (y * dy).sum() + (h * dh).sum()

    by_differences(loss, [x[n] for n in names],
                   [grads["d" + n] for n in names], 24)
