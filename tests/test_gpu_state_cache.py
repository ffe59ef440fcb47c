"""The quantised state cache on the GPU against the float64 definitions.  Codes,
scales and restored values are defined to the bit (one rounding each), so they
are compared for equality; what a run of decode steps loses by a stay in the
cache is bounded by the formats' own steps."""
import numpy as np
import pytest
import torch

import oracle.sanatan_oracle as O
import oracle.state_oracle as R
from constant_state_recurrence_gb300 import sanatan as S
from constant_state_recurrence_gb300 import workloads as W
from gpu_util import dev, f64, to_dev

pytestmark = pytest.mark.gpu

DT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def states(layers, B, inner, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(layers, B, inner, generator=gen)
    rows = torch.exp(2 * torch.randn(layers, B, -(-inner // 64), generator=gen))
    return x * rows.repeat_interleave(64, -1)[..., :inner]


def same(got, want):
    a, b = f64(got), np.asarray(want, dtype=np.float64)
    return a.shape == b.shape and np.array_equal(a, b, equal_nan=True)


def code_values(codes):
    return codes.to(torch.float32)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("layers,B,inner,zi", [
    (1, 1, 1, 0), (1, 3, 5, 1), (2, 2, 63, 3), (1, 4, 64, 4), (3, 5, 65, 0), (2, 3, 1000, 7),
    (1, 2, 384 * 64, 384), (2, 4, 640 * 64, 640), (12, 3, 1028, 5), (1, 300, 70, 2)])
def test_round_trip_to_the_bit(fmt, layers, B, inner, zi):
    x = states(layers, B, inner, inner + B)
    z = torch.rand(layers, B, zi) if zi else None
    P = B + 3
    pages = torch.randperm(P, generator=torch.Generator().manual_seed(B))[:B]
    codes, scales, zc = S.state_cache_empty(P, inner, zi, layers, DT[fmt])
    xd, zd, pd = x.to(dev()), None if z is None else z.to(dev()), pages.to(dev())
    S.sanatan_state_cache_write(xd, pd, codes, scales, zd, zc, layers)
    out = torch.full((layers, B, inner), -7.0, device=dev())
    zo = torch.full((layers, B, zi), -7.0, device=dev()) if zi else None
    S.sanatan_state_cache_read(codes, scales, pd, out, zc, zo, layers)
    torch.cuda.synchronize()
    c, s = R.cache_store(f64(x), fmt)                       # [layers, B, groups(, 64)]
    assert same(code_values(codes)[pages].transpose(0, 1), c)
    assert same(scales.cpu()[pages].transpose(0, 1), s)
    assert same(out, R.cache_values(c, s, inner))
    free = [p for p in range(P) if p not in pages.tolist()]
    assert not code_values(codes)[free].any() and not scales[free].any()
    if zi:
        assert torch.equal(zo, zd) and not zc[free].any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_values_next_to_borders(fmt):
    """Values that lie at, or one float32 step beside, the border between two codes,
    for many scales."""
    rng = np.random.default_rng(3)
    n = 4000
    top = np.float32(10.0 ** rng.uniform(-20, 20, n))
    x = np.zeros((n, 64), np.float32)
    x[:, 0] = top
    if fmt == "int8":
        s = np.float32(top.astype(np.float64) / 127).astype(np.float64)
        mid = rng.integers(-127, 127, (n, 21)) + 0.5
    else:
        _, s = R.cache_store(x, fmt)
        s = s[:, 0]
        mid = rng.integers(8, 16, (n, 21)) + 0.5
        mid = mid * 2.0 ** rng.integers(-9, 4, (n, 21)) * rng.choice([-1, 1], (n, 21))
    at = np.float32(mid * s[:, None])
    x[:, 1:22] = at
    x[:, 22:43] = np.nextafter(at, np.float32(np.inf))
    x[:, 43:64] = np.nextafter(at, np.float32(-np.inf))
    x = np.clip(x, -top[:, None], top[:, None])
    xt = torch.tensor(x).reshape(1, n, 64)
    codes, scales, _ = S.state_cache_empty(n, 64, dtype=DT[fmt])
    pages = torch.arange(n, device=dev())
    S.sanatan_state_cache_write(xt.to(dev()), pages, codes, scales)
    c, s = R.cache_store(x, fmt)
    assert same(scales[:, 0, 0], s[:, 0])
    assert same(code_values(codes)[:, 0, 0], c[:, 0])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_zeros_extremes_and_broken_groups(fmt):
    big, small = np.float32(1.7e38), np.float32(2.0 ** -99)
    x = np.zeros((10, 64), np.float32)
    x[1, 5] = big
    x[2] = -big
    x[3, 7] = small
    x[4, 8] = 2.0 ** -101
    x[5, 9] = np.inf
    x[6, 10] = np.nan
    x[7] = -0.0
    x[8, 11] = 3.4e38       # 2^127 and more: a code times its scale could overflow
    x[9, 12] = -1.7e38
    xd = torch.tensor(x).reshape(1, 1, 640).to(dev())
    codes, scales, _ = S.state_cache_empty(1, 640, dtype=DT[fmt])
    page = torch.zeros(1, dtype=torch.int64, device=dev())
    S.sanatan_state_cache_write(xd, page, codes, scales)
    out = torch.zeros_like(xd)
    S.sanatan_state_cache_read(codes, scales, page, out)
    c, s = R.cache_store(x.reshape(1, 640), fmt)
    assert same(scales[0, 0], s[0]) and same(out[0], R.cache_values(c, s, 640))
    assert torch.isnan(out[0, 0, 320:448]).all() and torch.isnan(out[0, 0, 512:576]).all()
    assert torch.isfinite(out[0, 0, :320]).all() and torch.isfinite(out[0, 0, 576:]).all()


def test_sequences_left_out_and_pages_named_twice():
    """Pages outside the pool leave sequence and pool alone; a page that a write
    names twice holds the last of the two, whole; reads may name one twice."""
    B, inner, P = 6, 640, 4
    x = states(1, B, inner, 5).to(dev())
    z = torch.rand(1, B, 10, device=dev())
    codes, scales, zc = S.state_cache_empty(P, inner, 10)
    pages = torch.tensor([2, -1, 0, 2, P, 1 << 40], device=dev())
    S.sanatan_state_cache_write(x, pages, codes, scales, z, zc)
    alone = S.state_cache_empty(P, inner, 10)
    S.sanatan_state_cache_write(x[:, 2:4].contiguous(), torch.tensor([0, 2], device=dev()),
                                *alone[:2], z[:, 2:4].contiguous(), alone[2])
    assert torch.equal(codes, alone[0]) and torch.equal(scales, alone[1])
    assert torch.equal(zc, alone[2]) and not scales[1].any() and not scales[3].any()
    out = torch.full((1, B, inner), 5.0, device=dev())
    zo = torch.full((1, B, 10), 5.0, device=dev())
    S.sanatan_state_cache_read(codes, scales, pages, out, zc, zo)
    assert torch.equal(out[0, 0], out[0, 3]) and torch.equal(zo[0, 0], z[0, 3])
    for b in (1, 4, 5):
        assert (out[0, b] == 5).all() and (zo[0, b] == 5).all()


def test_a_page_named_by_many_sequences_of_one_write():
    B, inner = 700, 130
    x = states(1, B, inner, 6).to(dev())
    codes, scales, _ = S.state_cache_empty(1, inner)
    S.sanatan_state_cache_write(x, torch.zeros(B, dtype=torch.int64, device=dev()), codes, scales)
    c, s = R.cache_store(f64(x[0, -1:]), "int8")
    assert same(code_values(codes)[0], c) and same(scales[0], s)


def test_layered_states_keep_their_order():
    """The stack decode's [L, B * heads, 6d, dv] order: layers = L."""
    L, B, heads = 3, 2, 4
    Sx = torch.randn(L, B * heads, 384, 64, generator=torch.Generator().manual_seed(1)).to(dev())
    z = torch.rand(L, B * heads, 384, device=dev())
    codes, scales, zc = S.state_cache_empty(5, heads * 384 * 64, heads * 384, layers=L)
    S.sanatan_state_cache_write(Sx, torch.tensor([4, 1], device=dev()), codes, scales, z, zc, L)
    So, zo = torch.zeros_like(Sx), torch.zeros_like(z)
    # taken up in the other order of sequences
    S.sanatan_state_cache_read(codes, scales, torch.tensor([1, 4], device=dev()), So, zc, zo, L)
    swap = lambda t: t.view(L, B, heads, *t.shape[2:]).flip(1).reshape(t.shape)  # noqa: E731
    assert torch.equal(zo, swap(z))
    # s / 2 with s = max|x| / 127 (1 + 2^-24), and the product c s rounded to float32:
    # max|x| / 254 (1 + 2^-24) + 2^-24 max|x| (1 + 2^-23) <= max|x| / 254 (1 + 256 2^-24);
    # the test's own subtraction and division add 2 steps of their values
    step = Sx.abs().amax(-1, keepdim=True) / 254
    assert ((swap(So) - Sx).abs() <= step * (1 + 260 * 2.0 ** -24)).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_prefill_park_resume_decode(fmt):
    """A prefilled sequence is put away, taken up into the slots of two sequences and
    decoded: the outputs are the formula's on the stored state (decode bar 1e-5), and
    off those of the unquantised state by no more than the stored rows are."""
    x = W.make(W.LAYER, B=1, H=3, T=200)
    g = to_dev(x)
    _, _, Sf, zf = S.sanatan_chunk_fwd(g["q"], g["k"], g["v"], g["gamma"], g["omega"], g["phi"],
                                       want_state=True)
    inner = 3 * 384 * 64
    codes, scales, zc = S.state_cache_empty(2, inner, 3 * 384, dtype=DT[fmt])
    S.sanatan_state_cache_write(Sf, torch.ones(1, dtype=torch.int64, device=dev()), codes, scales,
                                zf, zc)
    Sd = torch.empty(6, 384, 64, device=dev())
    zd = torch.empty(6, 384, device=dev())
    S.sanatan_state_cache_read(codes, scales, torch.ones(2, dtype=torch.int64, device=dev()), Sd,
                               zc, zd)
    kept = f64(Sd)
    assert np.array_equal(kept[:3], kept[3:]) and torch.equal(zd[:3], zf[0])
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(6, 64, generator=gen) for _ in range(3))
    pos = torch.full((6,), 200, dtype=torch.int64)
    o = S.sanatan_decode_step(Sd, zd, *(t.to(dev()) for t in (q, k, v)), g["gamma"], g["omega"],
                              g["phi"], pos.to(dev()))
    two = lambda t: np.concatenate([f64(t[0])] * 2)  # noqa: E731
    pars = [np.concatenate([f64(x[n])] * 2) for n in ("gamma", "omega", "phi")]
    args = (f64(q), f64(k), f64(v), *pars, f64(pos))
    _, _, stored = O.decode_step(kept, two(zf), *args)
    _, z1, exact = O.decode_step(two(Sf), two(zf), *args)
    assert np.abs(f64(o) - stored).max() <= 1e-5
    # |o - o'| <= sum_f |Phi_f| |S_f - S'_f| / D, with |S_f - S'_f| <= max|S_f| / 254 (int8) or
    # 2^-4 |S_f| + 2^-10 s, s <= max|S_f| / 224 (e4m3)
    top = np.abs(two(Sf)).max(-1, keepdims=True)
    off = top / 254 + 0 * two(Sf) if fmt == "int8" else np.abs(two(Sf)) / 16 + top / 224 / 1024
    phi = O.featurize(f64(q)[None, :, None], *pars, pos0=200)[0, :, 0]
    D = (phi * z1).sum(-1, keepdims=True)
    room = (np.abs(phi)[..., None] * off).sum(1) / D
    assert (np.abs(f64(o) - exact) <= room * (1 + 1e-3) + 1e-5).all()


def test_gated_recurrence_states_are_kept_too():
    """h [B, D] of the gated recurrence: scan, park, resume into steps."""
    x = torch.randn(2, 90, 771, device=dev())
    g = torch.randn(2, 90, 771, device=dev())
    _, h, _ = S.sanatan_gated_scan_fwd(x, g, "sigmoid", want_state=True)
    codes, scales, _ = S.state_cache_empty(3, 771)
    pages = torch.tensor([2, 0], device=dev())
    S.sanatan_state_cache_write(h, pages, codes, scales)
    back = torch.empty_like(h)
    S.sanatan_state_cache_read(codes, scales, pages, back)
    c, s = R.cache_store(f64(h), "int8")
    assert same(back, R.cache_values(c, s, 771))
    xt, gt = torch.randn(2, 771, device=dev()), torch.randn(2, 771, device=dev())
    ref = R.gated_scan_step(f64(back), f64(xt), f64(gt), "sigmoid")
    y = S.sanatan_gated_scan_step(back, xt, gt, "sigmoid")
    assert np.abs(f64(y) - ref).max() <= 20 * 2.0 ** -24 * (np.abs(f64(xt)) + np.abs(f64(h))).max()


def test_captured_park_and_resume():
    x = states(1, 3, 2000, 7).to(dev())
    codes, scales, _ = S.state_cache_empty(4, 2000)
    pages = torch.tensor([3, 1, 0], device=dev())
    out = torch.zeros_like(x)

    def both():
        S.sanatan_state_cache_write(x, pages, codes, scales)
        S.sanatan_state_cache_read(codes, scales, pages, out)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    new = states(1, 3, 2000, 8)
    x.copy_(new)
    pages.copy_(torch.tensor([2, 0, -1]))
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    c, s = R.cache_store(f64(new), "int8")
    want = R.cache_values(c, s, 2000)
    want[:, 2] = 0
    assert same(out, want)


def test_pools_beyond_32_bits():
    """A pool whose last page starts beyond 2^32 codes."""
    inner = 1 << 20
    P = 4200
    codes, scales, _ = S.state_cache_empty(P, inner)
    x = states(1, 2, inner, 9).to(dev())
    pages = torch.tensor([P - 1, 4097], device=dev())
    S.sanatan_state_cache_write(x, pages, codes, scales)
    out = torch.zeros_like(x)
    S.sanatan_state_cache_read(codes, scales, pages, out)
    c, s = R.cache_store(f64(x), "int8")
    assert same(out, R.cache_values(c, s, inner))
    assert not codes[:4097].any() and not codes[4098:P - 1].any()


def test_refusals_of_the_binding():
    x = torch.zeros(1, 2, 128, device=dev())
    pages = torch.zeros(2, dtype=torch.int64, device=dev())
    codes, scales, zc = S.state_cache_empty(3, 128, 4)
    z = torch.zeros(1, 2, 4, device=dev())
    W_ = S.sanatan_state_cache_write
    for bad in ((x[..., :100], pages, codes, scales), (x.to(torch.bfloat16), pages, codes, scales),
                (x, pages.to(torch.int32), codes, scales),
                (x, pages, codes.to(torch.uint8), scales),
                (x, pages, codes[:, :, :1], scales), (x, pages, codes, scales[:2]),
                (x, pages, codes, scales, z), (x, pages, codes, scales, z, zc[..., :3]),
                (x, pages, codes, scales, z, zc, 2), (x, pages, codes, scales, z, zc, 0),
                (x, pages.cpu(), codes, scales), (x[:, :, ::2], pages, codes, scales)):
        with pytest.raises(ValueError):
            W_(*bad)
    with pytest.raises(ValueError):
        S.sanatan_state_cache_read(codes, scales, pages, x[:, :1].expand(1, 2, 128))


def test_pages_out_of_a_longer_list():
    """pages[1:2], one sequence of a batch's list, starts at 8 bytes, not at 16."""
    x = states(1, 1, 640, 10).to(dev())
    codes, scales, _ = S.state_cache_empty(3, 640)
    pages = torch.tensor([0, 2, 1], device=dev())
    assert pages[1:2].data_ptr() % 16 == 8
    S.sanatan_state_cache_write(x, pages[1:2], codes, scales)
    out = torch.zeros_like(x)
    S.sanatan_state_cache_read(codes, scales, pages[1:2], out)
    c, s = R.cache_store(f64(x), "int8")
    assert same(out, R.cache_values(c, s, 640)) and same(scales[2], s[0, 0][None])
    assert not scales[:2].any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("inner,zi", [(771, 5), (640, 7), (3, 1), (24576, 384)])
def test_states_at_any_float(fmt, inner, zi):
    """One sequence's state and z out of a batch's."""
    x, z = states(1, 1, inner, 11), torch.rand(zi)
    at = lambda n: torch.full((n + 1,), 3.0, device=dev())  # noqa: E731
    xs, zs, xo, zo = at(inner), at(zi), at(inner), at(zi)
    xs[1:] = x.flatten().to(dev())
    zs[1:] = z.to(dev())
    codes, scales, zc = S.state_cache_empty(2, inner, zi, dtype=DT[fmt])
    page = torch.ones(1, dtype=torch.int64, device=dev())
    S.sanatan_state_cache_write(xs[1:].view(1, inner), page, codes, scales, zs[1:].view(1, zi), zc)
    S.sanatan_state_cache_read(codes, scales, page, xo[1:].view(1, inner), zc, zo[1:].view(1, zi))
    c, s = R.cache_store(f64(x), fmt)
    assert same(code_values(codes)[1, 0], c[0, 0]) and same(scales[1, 0], s[0, 0])
    assert same(xo[1:], R.cache_values(c, s, inner)[0, 0]) and torch.equal(zo, zs)
    assert xo[0] == 3 and not scales[0].any() and not zc[0].any()
    assert not code_values(codes)[0].any()


def gpu_ms(call, times=5):
    """The shortest of some runs, in milliseconds on the device."""
    ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
          for _ in range(times)]
    for a, b in ev:
        a.record()
        call()
        b.record()
    torch.cuda.synchronize()
    return min(a.elapsed_time(b) for a, b in ev[1:])


def test_sequences_left_out_are_not_read():
    """In the layered order one sequence is put away by naming the others -1: that does not
    take the time of reading them all.  Writing moves 4 + 1 + 4/64 bytes a value (1.3 GB
    here), of which reading is 4/5.06 = 0.79; blocks that do nothing stay well below half."""
    layers, B, inner = 12, 40, 1 << 19
    x = torch.ones(layers, B, inner, device=dev())
    codes, scales, _ = S.state_cache_empty(B, inner, layers=layers)
    pages = torch.arange(B, device=dev())
    none = torch.full_like(pages, -1)
    every = gpu_ms(lambda: S.sanatan_state_cache_write(x, pages, codes, scales, layers=layers))
    left = gpu_ms(lambda: S.sanatan_state_cache_write(x, none, codes, scales, layers=layers))
    assert left < every / 2, (left, every)


@pytest.mark.parametrize("layers", [1, 3])
def test_pages_named_again_much_later_in_a_large_write(layers):
    """Thousands of sequences in one write, most pages named twice, near and far: the last
    of the call's sequences is kept, whole."""
    B, inner, zi = 9001, 70, 3
    x = states(layers, B, inner, 12).to(dev())
    z = torch.rand(layers, B, zi, device=dev())
    gen = torch.Generator().manual_seed(13)
    pages = torch.randint(-1, 5000, (B,), generator=gen)
    pages[-1] = pages[0] = 17
    codes, scales, zc = S.state_cache_empty(5000, inner, zi, layers)
    S.sanatan_state_cache_write(x, pages.to(dev()), codes, scales, z, zc, layers)
    last = {p: b for b, p in enumerate(pages.tolist()) if p >= 0}
    named = torch.tensor(sorted(last))
    at = torch.tensor([last[p] for p in named.tolist()])
    c, s = R.cache_store(f64(x)[:, at.numpy()], "int8")
    assert same(code_values(codes)[named].transpose(0, 1), c)
    assert same(scales.cpu()[named].transpose(0, 1), s)
    assert torch.equal(zc[named.to(dev())].transpose(0, 1), z[:, at.to(dev())])
    free = torch.ones(5000, dtype=torch.bool)
    free[named] = False
    assert not scales.cpu()[free].any() and not code_values(codes)[free.to(dev())].any()


def test_writes_take_time_in_proportion_to_their_sequences():
    """Eight times the (small) sequences: not 64 times the time."""
    def ms(B):
        x = torch.ones(B, 64, device=dev())
        codes, scales, _ = S.state_cache_empty(B, 64)
        pages = torch.arange(B, device=dev())
        return gpu_ms(lambda: S.sanatan_state_cache_write(x, pages, codes, scales))

    small, large = ms(1 << 15), ms(1 << 18)
    assert large < 20 * small, (small, large)


def test_captured_large_write():
    """A write of several launches in a graph, replayed on other states and pages."""
    B, inner = 7000, 66
    x = states(1, B, inner, 14).to(dev())
    pages = torch.arange(B, device=dev()) % 3000
    pool = S.state_cache_empty(3000, inner)[:2]
    S.sanatan_state_cache_write(x, pages, *pool)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.sanatan_state_cache_write(x, pages, *pool)
    x.mul_(-3)
    pages.copy_(pages.flip(0).clone())
    graph.replay()
    torch.cuda.synchronize()
    want = S.state_cache_empty(3000, inner)[:2]
    S.sanatan_state_cache_write(x, pages, *want)
    assert torch.equal(pool[0], want[0]) and torch.equal(pool[1], want[1])
    c, s = R.cache_store(f64(x[0, -1000:]), "int8")      # nobody names these again
    assert same(code_values(pool[0])[pages[-1000:]][:, 0], c)
