"""Layer norm, short convolution, selective scan and the state cache as a layer of a small
model uses them: trained by one backward through all three, on halves of the layer's
projections and beside a residual stream; and served: a padded batch of prompts, its states
put away, taken up in another order, and decoded token by token."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as R
import oracle.state_oracle as C
from constant_state_recurrence_gb300 import sanatan as S
from gpu_util import dev, f64, rel_fro

pytestmark = pytest.mark.gpu

M, D, N, K, RANK = 24, 48, 16, 4, 3     # model width, channels, states, taps, rank of dt


def weights(seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    size = torch.exp(torch.rand(D, generator=gen) * 4.6 - 6.9)
    return dict(norm_w=1 + 0.2 * n(M), norm_b=0.1 * n(M), w_in=n(M, 2 * D) / M ** 0.5,
                conv_w=n(D, K) / 2, conv_b=0.2 * n(D), w_x=n(D, RANK + 2 * N) / D ** 0.5,
                w_dt=n(RANK, D) / RANK ** 0.5, dt_bias=size + torch.log(-torch.expm1(-size)),
                A=-(torch.arange(N) + 1.0) * torch.exp(0.1 * n(D, N)), skip=1 + 0.1 * n(D),
                w_out=n(D, M) / D ** 0.5)


def inputs(B, T, seed):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(B, T, M, generator=gen) for _ in range(4)]


def layer(p, x, residual):
    """The layer on the library's entry points: (output, stream)."""
    y, stream = S.LayerNorm.apply(x, p["norm_w"], p["norm_b"], residual)
    both = y @ p["w_in"]
    u, _ = S.CausalConv.apply(both[..., :D], p["conv_w"], p["conv_b"], "silu")
    rows = u @ p["w_x"]
    dt = rows[..., :RANK] @ p["w_dt"]
    y, _ = S.SelectiveScan.apply(u, dt, p["A"], rows[..., RANK:RANK + N], rows[..., RANK + N:],
                                 p["skip"], both[..., D:], p["dt_bias"])
    return y @ p["w_out"], stream


def layer_64(p, x, residual):
    """The same from elementary operations, token by token."""
    stream = x + residual
    far = stream - stream.mean(-1, keepdim=True)
    y = far / (far.square().mean(-1, keepdim=True) + 1e-5).sqrt() * p["norm_w"] + p["norm_b"]
    both = y @ p["w_in"]
    B, T, _ = x.shape
    before = torch.cat([both.new_zeros(B, K - 1, D), both[..., :D]], 1)
    c = p["conv_b"] + sum(p["conv_w"][:, k] * before[:, k:k + T] for k in range(K))
    u = c * torch.sigmoid(c)
    rows = u @ p["w_x"]
    delta = torch.log1p(torch.exp(rows[..., :RANK] @ p["w_dt"] + p["dt_bias"]))
    h, out = both.new_zeros(B, D, N), []
    for t in range(T):
        h = torch.exp(delta[:, t, :, None] * p["A"]) * h \
            + (delta[:, t] * u[:, t])[..., None] * rows[:, t, None, RANK:RANK + N]
        out.append((h * rows[:, t, None, RANK + N:]).sum(-1) + p["skip"] * u[:, t])
    z = both[..., D:]
    return (torch.stack(out, 1) * z * torch.sigmoid(z)) @ p["w_out"], stream


@pytest.mark.parametrize("B,T", [(2, 40), (1, 150)])
def test_one_backward_through_all(B, T):
    """Values and gradients against autograd in float64, 1e-4 of a tensor's norm: the three
    operators are within some 1e-6 each, the projections, sums of at most 48 products, within
    3e-6 of theirs, and a gradient passes ten of them."""
    p, (x, r, wy, ws) = weights(1), inputs(B, T, 2)
    ref = {n: t.double().requires_grad_() for n, t in p.items()}
    xr, rr = x.double().requires_grad_(), r.double().requires_grad_()
    y64, s64 = layer_64(ref, xr, rr)
    ((y64 * wy.double()).sum() + (s64 * ws.double()).sum()).backward()
    on = {n: t.to(dev()).requires_grad_() for n, t in p.items()}
    xd, rd = x.to(dev()).requires_grad_(), r.to(dev()).requires_grad_()
    y, s = layer(on, xd, rd)
    ((y * wy.to(dev())).sum() + (s * ws.to(dev())).sum()).backward()
    assert rel_fro(f64(y), y64.detach().numpy()) <= 1e-4
    assert rel_fro(f64(s), s64.detach().numpy()) <= 1e-6
    for n in p:
        assert rel_fro(f64(on[n].grad), ref[n].grad.numpy()) <= 1e-4, n
    assert rel_fro(f64(xd.grad), xr.grad.numpy()) <= 1e-4
    assert torch.equal(xd.grad, rd.grad)


def serve_64(p, x, conv, h):
    """One token of every sequence in float64 from the states: (y, conv, h)."""
    y = R.layer_norm(x, p["norm_w"], p["norm_b"])[0] @ p["w_in"]
    u, conv, _ = R.causal_conv(y[:, None, :D], p["conv_w"], p["conv_b"], s0=conv)
    rows = u[:, 0] @ p["w_x"]
    out, h, _ = R.selective_scan(u, (rows[:, :RANK] @ p["w_dt"])[:, None], p["A"],
                                 rows[:, None, RANK:RANK + N], rows[:, None, RANK + N:], p["skip"],
                                 y[:, None, D:], p["dt_bias"], h0=h)
    return out[:, 0] @ p["w_out"], conv, h


@pytest.mark.parametrize("dtype,name", [(torch.int8, "int8"), (torch.float8_e4m3fn, "e4m3")])
def test_prefill_put_away_take_up_decode(dtype, name):
    """The scan's state in 8 bits, the convolution's beside it in float32, both in one page.
    Against float64 from the states as the cache holds them; bar 1e-4 as above."""
    B, T = 3, 37
    p, lens = weights(3), [37, 12, 2]
    on = {n: t.to(dev()) for n, t in p.items()}
    n64 = {n: f64(t) for n, t in p.items()}
    x = inputs(B, T + 3, 4)[0]
    ln = torch.tensor(lens, device=dev())
    y, _, _ = S.sanatan_layer_norm_fwd(x[:, :T].contiguous().to(dev()), on["norm_w"], on["norm_b"])
    both = y @ on["w_in"]
    u, conv = S.sanatan_causal_conv_fwd(both[..., :D], on["conv_w"], on["conv_b"], lens=ln,
                                        want_state=True)
    rows = u @ on["w_x"]
    args = dict(D=on["skip"], dt_bias=on["dt_bias"])
    _, h, _ = S.sanatan_selective_scan_fwd(
        u, rows[..., :RANK] @ on["w_dt"], on["A"], rows[..., RANK:RANK + N], rows[..., RANK + N:],
        z=both[..., D:], lens=ln, want_state=True, **args)
    # each sequence's states are those of its own tokens alone
    for b, n in enumerate(lens):
        c64, h64 = np.zeros((1, K - 1, D)), np.zeros((1, D, N))
        for t in range(n):
            _, c64, h64 = serve_64(n64, f64(x[b:b + 1, t]), c64, h64)
        assert rel_fro(f64(conv[b]), c64[0]) <= 1e-4 and rel_fro(f64(h[b]), h64[0]) <= 1e-4
    codes, scales, exact = S.state_cache_empty(5, D * N, (K - 1) * D, dtype=dtype, device=dev())
    pages = torch.tensor([4, 0, 2], device=dev())
    S.sanatan_state_cache_write(h, pages, codes, scales, conv, exact)
    order = [2, 0, 1]
    h2, conv2 = torch.zeros_like(h), torch.zeros_like(conv)
    S.sanatan_state_cache_read(codes, scales, pages[order].contiguous(), h2, exact, conv2)
    held = C.cache_values(*C.cache_store(f64(h).reshape(B, -1), name), D * N)[order]
    assert np.array_equal(f64(h2).reshape(B, -1), held) and torch.equal(conv2, conv[order])
    c64, h64 = f64(conv2), held.reshape(B, D, N)
    for t in range(3):
        xt = x[order, T + t]
        y, _, _ = S.sanatan_layer_norm_fwd(xt.contiguous().to(dev()), on["norm_w"], on["norm_b"])
        both = y @ on["w_in"]
        u = S.sanatan_causal_conv_step(conv2, both[:, :D], on["conv_w"], on["conv_b"])
        rows = u @ on["w_x"]
        y = S.sanatan_selective_scan_step(h2, u, rows[:, :RANK] @ on["w_dt"], on["A"],
                                          rows[:, RANK:RANK + N], rows[:, RANK + N:],
                                          z=both[:, D:], **args) @ on["w_out"]
        want, c64, h64 = serve_64(n64, f64(xt), c64, h64)
        assert rel_fro(f64(y), want) <= 1e-4
    assert rel_fro(f64(h2), h64) <= 1e-4 and rel_fro(f64(conv2), c64) <= 1e-4


def test_the_layer_captured():
    """Forward and backward of the layer as one graph, replayed on other data."""
    p = {n: t.to(dev()).requires_grad_() for n, t in weights(5).items()}
    x, r, wy, _ = (t.to(dev()) for t in inputs(2, 60, 6))
    x.requires_grad_()
    leaves = [x] + list(p.values())

    def step():
        y, s = layer(p, x, r)
        return torch.autograd.grad((y * wy).sum() + s.sum(), leaves)

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
        p["A"].mul_(1.1)
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    for a, b in zip(got, want):     # (the projections may run on other kernels in a graph)
        assert rel_fro(f64(a), f64(b)) <= 1e-5
