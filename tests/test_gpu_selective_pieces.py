"""The selective scan's backward in pieces: more than 16 states and more than 512 MB of parts
of dB and dC.  A piece goes on from what the one behind it left, to the bit, so that gradients
are what calls of few sequences give; sequences cut into segments and pieces both are held
against the float64 definitions."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as R
from constant_state_recurrence_gb300 import sanatan as S
from gpu_util import dev, f64
from test_gpu_layer_norm import BF16, F32, close
from test_gpu_selective_scan import bounds, make

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
MOST = 1 << 29


def parts(b, T, D, N):
    """Bytes of all parts of dB and dC."""
    lanes = 8 if N <= 32 else 16 if N <= 64 else 32
    return -(-D * lanes // 128) * b * T * 2 * N * 4


def grads(x, dy, dh, lens=None):
    d = dict(x)
    h0 = d.pop("h0")
    _, _, marks = S.sanatan_selective_scan_fwd(**d, h0=h0, lens=lens, want_marks=True)
    return S.sanatan_selective_scan_bwd(**d, dy=dy, marks=marks, lens=lens, dh_last=dh,
                                        want_dh0=True)


@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (F32, 63)])
def test_segments_in_pieces(dtype, D):
    """1500 tokens of 132000: two segments of 1168, of two pieces each; what is behind the last
    token is NaN and has no effect."""
    T, n, N = 132000, 1500, 64
    assert parts(1, T, D, N) > MOST
    x, dy, dh = make(1, n, D, N, dtype, D)

    def long(t):
        out = torch.full((1, T, t.shape[2]), float("nan"), dtype=t.dtype, device=dev())
        out[:, :n] = t.to(dev())
        return out
    row = ("u", "dt", "B", "C", "z")
    d = {k: long(t) if k in row else t.to(dev()) for k, t in x.items()}
    ln = torch.tensor([n], device=dev())
    g = grads(d, long(dy), dh.to(dev()), ln)
    v = {k: f64(t) for k, t in x.items()}
    ref = R.selective_scan_backward(**v, dy=f64(dy), dh_last=f64(dh))
    bd = bounds(v, True, None, f64(dy), f64(dh))
    for k in ("du", "ddt", "dz", "dB", "dC"):
        assert not g[k][:, n:].any(), k
        close(g[k][:, :n], ref[k], bd[k] + 1e-34, dtype, k)
    for k in ("dA", "dD", "ddt_bias", "dh0"):
        close(g[k], ref[k], bd[k] + 1e-34, F32, k)
    again = grads(d, long(dy), dh.to(dev()), ln)
    assert all(torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("lens,N,dtype", [(None, 128, F32), ([2100, 0, 700, 1], 128, F32),
                                          ([2100, 2099, 701, 16], 127, BF16)])
def test_whole_sequences_in_pieces(lens, N, dtype):
    """Four sequences in three pieces are four of one, to the bit; sums over sequences are
    formed in their order."""
    b, T, D = 4, 2100, 512
    assert parts(b, T, D, N) > 2 * MOST > MOST > parts(1, T, D, N)
    x, dy, dh = make(b, T, D, N, dtype, 11)
    x = {k: t.to(dev()) for k, t in x.items()}
    dy, dh = dy.to(dev()), dh.to(dev())
    ln = None if lens is None else torch.tensor(lens, device=dev())
    g = grads(x, dy, dh, ln)
    many = ("u", "dt", "B", "C", "z", "h0")
    total = {}
    for i in range(b):
        one = grads({k: t[i:i + 1] if k in many else t for k, t in x.items()}, dy[i:i + 1],
                    dh[i:i + 1], None if ln is None else ln[i:i + 1])
        for k in ("du", "ddt", "dz", "dB", "dC", "dh0"):
            assert torch.equal(g[k][i:i + 1], one[k]), (k, i)
        for k in ("dA", "dD", "ddt_bias"):
            total[k] = one[k] if i == 0 else total[k] + one[k]
    assert all(torch.equal(g[k], total[k]) for k in total)


def test_two_pieces_of_eight_lanes():
    """Ten sequences in two pieces, five in one.  dA and dD are sums of ten values of one sign,
    in another order: 15 roundings at most; ddt_bias as many of the sum of |ddt|, itself rounded
    to bf16."""
    b, T, D, N = 10, 4200, 1024, 32
    assert parts(b, T, D, N) > MOST > parts(5, T, D, N)
    x, dy, dh = make(b, T, D, N, BF16, 12, gated=False)
    x = {k: None if t is None else t.to(dev()) for k, t in x.items()}
    for k in ("u", "B", "C", "D", "h0"):
        x[k] = x[k].abs()
    dy, dh = dy.to(dev()).abs(), dh.to(dev()).abs()
    many = ("u", "dt", "B", "C", "h0")
    g = grads(x, dy, dh)
    half = [grads({k: t[p] if k in many else t for k, t in x.items()}, dy[p], dh[p])
            for p in (slice(0, 5), slice(5, 10))]
    for k in ("du", "ddt", "dB", "dC", "dh0"):
        assert torch.equal(g[k], torch.cat([h[k] for h in half])), k
    for k in ("dA", "dD"):
        want = f64(half[0][k]) + f64(half[1][k])
        assert (np.abs(f64(g[k]) - want) <= 15 * E * want).all(), k
    want = f64(half[0]["ddt_bias"]) + f64(half[1]["ddt_bias"])
    room = 15 * E * (1 + 2.0 ** -8) * np.abs(f64(g["ddt"])).sum((0, 1))
    assert (np.abs(f64(g["ddt_bias"]) - want) <= room).all()
