"""The two constant-state mixers and the state cache as a small model uses them: a
layer of p = 1 attention whose outputs a layer of the gated recurrence mixes, trained
by one backward through both, and served: prefilled, put away, taken up in another
batch order and decoded token by token."""
import numpy as np
import pytest
import torch

import oracle.sanatan_oracle as O
import oracle.state_oracle as R
from constant_state_recurrence_gb300 import sanatan as S
from constant_state_recurrence_gb300 import workloads as W
from gpu_util import dev, f64, rel_fro, to_dev

pytestmark = pytest.mark.gpu

H, T = 2, 120
D = H * 64


def _inputs(B, seed):
    x = W.make(W.TINY, B=B, H=H, T=T)
    x["phi"] = W.rates(H, 64, "geometric")
    gen = torch.Generator().manual_seed(seed)
    gates = torch.randn(B, T + 4, D, generator=gen) + 1
    return x, gates, gen


def _flat(o):
    """Heads side by side: [B, H, T, 64] -> [B, T, H * 64]."""
    return o.transpose(1, 2).flatten(2)


def test_one_backward_through_both():
    """Gradients of sum(y w) in q, k, v, the gates and the attention's parameters, against
    the two formulas one after the other in float64 (attention bar 1e-4)."""
    x, gates, gen = _inputs(2, 1)
    g = {n: t.requires_grad_() for n, t in to_dev(x).items()}
    gt = gates[:, :T].contiguous().to(dev()).requires_grad_()
    w = torch.randn(2, T, D, generator=gen)
    o = S.SanatanAttention.apply(g["q"], g["k"], g["v"], g["gamma"], g["omega"], g["phi"])
    y, _ = S.GatedScan.apply(_flat(o).contiguous(), gt, "sigmoid")
    (y * w.to(dev())).sum().backward()
    ra = {n: f64(x[n]) for n in ("q", "k", "v", "gamma", "omega", "phi")}
    o_ref, _ = O.attn_quadratic(**ra)
    flat = o_ref.transpose(0, 2, 1, 3).reshape(2, T, D)
    dflat, dg, _ = R.gated_scan_backward(flat, f64(gates[:, :T]), "sigmoid", f64(w))
    ref = O.attn_backward(**ra, dO=dflat.reshape(2, T, H, 64).transpose(0, 2, 1, 3))
    assert rel_fro(f64(gt.grad), dg) <= 1e-4
    for n in ("q", "k", "v", "gamma", "omega"):
        assert rel_fro(f64(g[n].grad), ref["d" + n]) <= 1e-4, n


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_prefill_put_away_take_up_decode(fmt):
    """Against the same tokens in float64 from the states as the cache holds them: the
    attention within its decode bar of 1e-5, the recurrence, which mixes it, within that
    bar times 1 - a summed over the steps (at most the bar) and its own roundings."""
    B = 3
    x, gates, gen = _inputs(B, 2)
    g = to_dev(x)
    o, _, Sf, zf = S.sanatan_chunk_fwd(g["q"], g["k"], g["v"], g["gamma"], g["omega"], g["phi"],
                                       want_state=True)
    gd = gates.to(dev())
    _, h, _ = S.sanatan_gated_scan_fwd(_flat(o).contiguous(), gd[:, :T].contiguous(), "sigmoid",
                                       want_state=True)
    dt = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    pages = torch.tensor([4, 1, 2], device=dev())
    attn = S.state_cache_empty(5, H * 384 * 64, H * 384, dtype=dt)
    rec = S.state_cache_empty(5, D, dtype=dt)
    S.sanatan_state_cache_write(Sf, pages, attn[0], attn[1], zf, attn[2])
    S.sanatan_state_cache_write(h, pages, *rec[:2])
    order = [2, 0, 1, 0]                                # one sequence goes on twice
    take = pages[torch.tensor(order, device=dev())]
    n = len(order)
    Sd, zd = torch.empty(n * H, 384, 64, device=dev()), torch.empty(n * H, 384, device=dev())
    hd = torch.empty(n, D, device=dev())
    S.sanatan_state_cache_read(attn[0], attn[1], take, Sd, attn[2], zd)
    S.sanatan_state_cache_read(*rec[:2], take, hd)
    c, s = R.cache_store(f64(h), fmt)
    assert np.array_equal(f64(hd), R.cache_values(c, s, D)[order])
    Sr, zr, hr = f64(Sd), f64(zd), f64(hd)
    par = [np.concatenate([f64(x[p])] * n) for p in ("gamma", "omega", "phi")]
    for t in range(4):
        q, k, v = (torch.randn(n * H, 64, generator=gen) for _ in range(3))
        pos = torch.full((n * H,), T + t, dtype=torch.int64)
        od = S.sanatan_decode_step(Sd, zd, *(a.to(dev()) for a in (q, k, v)), g["gamma"],
                                   g["omega"], g["phi"], pos.to(dev()))
        gate = gd[order, T + t].contiguous()
        y = S.sanatan_gated_scan_step(hd, od.view(n, D), gate, "sigmoid")
        Sr, zr, o_ref = O.decode_step(Sr, zr, f64(q), f64(k), f64(v), *par, f64(pos))
        assert np.abs(f64(od) - o_ref).max() <= 1e-5
        hr = R.gated_scan_step(hr, o_ref.reshape(n, D), f64(gate), "sigmoid")
        size = max(np.abs(hr).max(), np.abs(o_ref).max())
        # 4 steps of at most (10 + 2 |g| + 3) 2^-24 of the largest value each
        room = 1e-5 + 4 * (13 + 2 * np.abs(f64(gate)).max()) * 2.0 ** -24 * size
        assert np.abs(f64(y) - hr).max() <= room, t
