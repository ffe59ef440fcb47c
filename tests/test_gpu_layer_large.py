"""Norm, short convolution and selective scan over tensors of more than 2^31 values: what the
last tokens give is what a call of these tokens alone gives (to the bit where every output is
formed by itself, else against float64 with the bounds of the small cases)."""
import pytest
import torch

import oracle.layer_oracle as R
import test_gpu_causal_conv as conv
import test_gpu_layer_norm as norm
import test_gpu_selective_scan as scan
from constant_state_recurrence_gb300 import sanatan as S
from gpu_util import dev, f64
from test_gpu_layer_norm import BF16, F32, close

pytestmark = pytest.mark.gpu

TAIL = 64


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def many(*shape, seed):
    gen = torch.Generator(device=dev()).manual_seed(seed)
    t = torch.randn(*shape, generator=gen, dtype=BF16, device=dev())
    assert t.numel() > 1 << 31
    return t


@pytest.mark.parametrize("D", [768, 771])
def test_rows(D):
    rows = (1 << 31) // D + 1000
    x = many(rows, D, seed=D)
    _, _, dy, _, w, b = (t.to(dev()) for t in norm.make(TAIL, D, BF16, 5))
    y, _, stats = S.sanatan_layer_norm_fwd(x, w, b, want_stats=True)
    last = x[-TAIL:].contiguous()
    y1, _, stats1 = S.sanatan_layer_norm_fwd(last, w, b, want_stats=True)
    assert torch.equal(y[-TAIL:], y1) and torch.equal(stats[-TAIL:], stats1)
    all_dy = y.zero_()
    all_dy[-TAIL:] = dy
    g = S.sanatan_layer_norm_bwd(x, w, all_dy, stats)
    one = S.sanatan_layer_norm_bwd(last, w, dy, stats1)
    assert torch.equal(g["dx"][-TAIL:], one["dx"]) and not g["dx"][:-TAIL].any()
    # (zeros add nothing, so that the sums are those of the last rows in another order)
    s, w, b, dy = f64(last), f64(w), f64(b), f64(dy)
    bd = norm.bounds(s, w, b, dy)
    _, dw, db = R.layer_norm_backward(s, w, dy)
    close(g["dweight"], dw, bd["dw"], F32, "dweight")
    close(g["dbias"], db, bd["db"], F32, "dbias")


def test_tokens_of_a_convolution():
    B, T, D, K = 2, 750_000, 1536, 4
    x = many(B, T, D, seed=1)
    _, w, bias, dy, _, _ = (t.to(dev()) for t in conv.make(1, TAIL, D, K, BF16, 2))
    y, s = S.sanatan_causal_conv_fwd(x, w, bias, want_state=True)
    last = x[-1:, -TAIL:].contiguous()
    s0 = x[-1:, -TAIL - K + 1:-TAIL].float().contiguous()
    y1, s1 = S.sanatan_causal_conv_fwd(last, w, bias, s0=s0, want_state=True)
    assert torch.equal(y[-1:, -TAIL:], y1) and torch.equal(s[-1:], s1)
    all_dy = y.zero_()
    all_dy[-1:, -TAIL:] = dy
    g = S.sanatan_causal_conv_bwd(x, w, all_dy, bias)
    n = [f64(t) for t in (last, w, dy, bias, s0)]
    dx, dw, db, _ = R.causal_conv_backward(n[0], n[1], n[2], n[3], True, n[4], None, None)
    bd = conv.bounds(n[0], n[1], n[3], True, n[4], None, n[2])
    close(g["dx"][-1:, -TAIL:], dx, bd["dx"], BF16, "dx")
    assert not g["dx"][0].any() and not g["dx"][-1, :-TAIL - K + 1].any()
    close(g["dw"], dw, bd["dw"], F32, "dw")
    close(g["dbias"], db, bd["dbias"], F32, "dbias")


def test_tokens_of_a_scan():
    B, T, D, N = 2, 750_000, 1536, 16
    t0 = T - TAIL
    assert t0 % S.SELECTIVE_MARK == 0
    x, dy, _ = scan.make(1, TAIL, D, N, BF16, 3)
    d = scan.on({k: x[k] for k in ("A", "D", "dt_bias")})
    for i, k in enumerate(("u", "dt", "z")):
        d[k] = many(B, T, D, seed=4 + i)
        if k == "dt":
            d[k].mul_(0.6)
        d[k][-1:, t0:] = x[k].to(dev())
    for k in ("B", "C"):
        d[k] = torch.randn(B, T, N, device=dev()).to(BF16)
        d[k][-1:, t0:] = x[k].to(dev())
    y, h, marks = S.sanatan_selective_scan_fwd(**d, want_state=True, want_marks=True)
    y1 = y[-1:, t0:].clone()
    all_dy = y.zero_()
    all_dy[-1:, t0:] = dy.to(dev())
    g = S.sanatan_selective_scan_bwd(**d, dy=all_dy, marks=marks)
    n = {k: f64(t) for k, t in x.items()}
    n["h0"] = f64(marks[-1:, t0 // S.SELECTIVE_MARK])
    y_ref, h_ref, _ = R.selective_scan(**n, soft=True, lens=None)
    ref = R.selective_scan_backward(**n, soft=True, lens=None, dy=f64(dy), dh_last=None)
    bd = scan.bounds(n, True, None, f64(dy))
    close(y1, y_ref, bd["y"] + 1e-34, BF16, "y")
    close(h[-1:], h_ref, bd["last"] + 1e-34, F32, "h_last")
    for k in ("du", "ddt", "dz", "dB", "dC"):
        close(g[k][-1:, t0:], ref[k], bd[k] + 1e-34, BF16, k)
        assert not g[k][0].any(), k
