"""Pins of the float64 definitions in oracle/state_oracle.py: closed forms,
finite differences, brute force over all codes; and the refusals of the gated
recurrence's and the state cache's entry points that need no GPU."""
import ctypes

import numpy as np
import pytest

import oracle.state_oracle as R


def _inputs(B, T, D, seed=0):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((B, T, D)), rng.standard_normal((B, T, D)) - 0.3,
            rng.standard_normal((B, D)))


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
def test_scan_is_the_sum_of_decayed_inputs(gate):
    """h_t = (prod a) h0 + sum_j (prod_{j<i<=t} a_i) u_j, term by term."""
    x, g, h0 = _inputs(2, 9, 3)
    a = np.exp(g) if gate == "log" else 1 / (1 + np.exp(-g))
    u = x if gate == "log" else (1 - a) * x
    y, last, _ = R.gated_scan(x, g, gate, h0)
    for t in range(9):
        want = np.prod(a[:, :t + 1], 1) * h0
        for j in range(t + 1):
            want = want + np.prod(a[:, j + 1:t + 1], 1) * u[:, j]
        assert np.abs(y[:, t] - want).max() <= 1e-12
    assert np.array_equal(last, y[:, -1])


def test_constant_gates_have_closed_forms():
    x = np.ones((1, 50, 1))
    g = np.full((1, 50, 1), np.log(0.9))
    y, _, _ = R.gated_scan(x, g, "log")
    assert np.abs(y[0, :, 0] - (1 - 0.9 ** np.arange(1, 51)) / 0.1).max() <= 1e-12
    y, _, _ = R.gated_scan(x * 3, g * 0 + 2.0, "sigmoid")      # a convex mean tends to its input
    a = 1 / (1 + np.exp(-2.0))
    assert np.abs(y[0, :, 0] - 3 * (1 - a ** np.arange(1, 51))).max() <= 1e-12


def test_a_closed_gate_starts_a_new_text_and_lengths_cut():
    x, g, h0 = _inputs(2, 12, 2, 3)
    g[:, 5] = -np.inf
    y, _, _ = R.gated_scan(x, g, "log", h0)
    z, _, _ = R.gated_scan(x[:, 5:], np.where(np.isinf(g[:, 5:]), 0.0, g[:, 5:]), "log")
    assert np.array_equal(y[:, 5:], z)
    y, last, _ = R.gated_scan(x, g, "log", h0, lens=[7, 0])
    full, _, _ = R.gated_scan(x, g, "log", h0)
    assert np.array_equal(y[0, :7], full[0, :7]) and not y[0, 7:].any() and not y[1].any()
    assert np.array_equal(last[0], full[0, 6]) and np.array_equal(last[1], h0[1])


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
def test_gradients_by_differences(gate):
    x, g, h0 = _inputs(2, 7, 2, 5)
    rng = np.random.default_rng(6)
    dy, dh = rng.standard_normal((2, 7, 2)), rng.standard_normal((2, 2))
    lens = [7, 4]

    def loss(x, g, h0):
        y, last, _ = R.gated_scan(x, g, gate, h0, lens)
        return (y * dy).sum() + (last * dh).sum()

    grads = R.gated_scan_backward(x, g, gate, dy, h0, lens, dh)
    args = [x, g, h0]
    for k in range(3):
        for i in np.ndindex(args[k].shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[k][i] += 1e-5
            down[k][i] -= 1e-5
            d = (loss(*up) - loss(*down)) / 2e-5
            assert abs(d - grads[k][i]) <= 1e-8 * (1 + abs(d)), (k, i)


def _e4m3_values():
    v = []
    for code in range(256):
        s, e, m = code >> 7, (code >> 3) & 15, code & 7
        if e == 15 and m == 7:
            continue
        x = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        v.append(-x if s else x)
    return np.unique(np.array(v))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_stored_values_are_the_nearest_ones(fmt):
    rng = np.random.default_rng(8)
    x = np.float32(rng.standard_normal((6, 64)) * 10.0 ** rng.uniform(-4, 4, (6, 1)))
    codes, s = R.cache_store(x, fmt)
    every = np.arange(-127, 128) if fmt == "int8" else _e4m3_values()
    for r in range(6):
        top = np.abs(x[r]).max().astype(np.float64)
        if fmt == "int8":
            assert abs(s[r] / (top / 127) - 1) <= 2.0 ** -24
        else:
            assert np.log2(s[r]) % 1 == 0 and 224 < top / s[r] <= 448
        near = np.abs(every[None] * s[r] - x[r].astype(np.float64)[:, None]).min(1)
        assert np.array_equal(np.abs(codes[r, 0] * s[r] - x[r]), near)
        assert np.isin(codes[r, 0], every).all()


def test_ties_go_to_even_codes():
    x = np.zeros(64)
    x[0] = 127.0
    x[1:6] = [0.5, 1.5, 2.5, -0.5, -3.5]
    codes, s = R.cache_store(x, "int8")
    assert s[0] == 1.0 and list(codes[0, 1:6]) == [0, 2, 2, 0, -4]
    assert R.e4m3_round(17.0) == 16.0 and R.e4m3_round(19.0) == 20.0
    assert R.e4m3_round(2.0 ** -10) == 0.0 and R.e4m3_round(3 * 2.0 ** -10) == 2.0 ** -8


def test_small_ragged_and_broken_groups():
    codes, s = R.cache_store(np.full(70, 2.0 ** -101), "int8")
    assert codes.shape == (2, 64) and not codes.any() and not s.any()
    x = np.ones(130)
    x[65] = np.inf
    codes, s = R.cache_store(x, "e4m3")
    assert np.isnan(s[1]) and s[0] == s[2] == 2.0 ** -8 and not codes[2, 2:].any()


@pytest.fixture(scope="module")
def lib():
    from constant_state_recurrence_gb300 import build, sanatan
    build.build(quiet=True)
    return sanatan.lib()


def test_scan_refusals(lib):
    """Every call here is refused on the host: one thing is wrong with each."""
    P = ctypes.c_void_p
    at = [P((i + 1) << 20) for i in range(9)]      # ranges that share nothing

    def fwd(x=at[0], g=at[1], dt=0, gate=0, lens=None, B=2, T=3, D=4, h0=None, y=at[2], h=None,
            m=None):
        return lib.sanatan_gated_scan_fwd(x, g, dt, gate, lens, B, T, D, h0, y, h, m, None)

    assert fwd(dt=2) == 1 and fwd(gate=2) == 1 and fwd(gate=-1) == 1
    assert fwd(B=-1) == 1 and fwd(T=-1) == 1 and fwd(D=-1) == 1
    assert fwd(x=None) == 1 and fwd(g=P(24)) == 1 and fwd(y=None) == 1
    assert fwd(lens=P(8)) == 1 and fwd(h0=P(4)) == 1 and fwd(h=P(8)) == 1 and fwd(m=P(8)) == 1
    assert fwd(B=1 << 20, D=1 << 11) == 2 and fwd(T=(1 << 30) + 1) == 2
    assert fwd(B=1, T=1, D=(1 << 30) + 1) == 2
    assert fwd(B=0) == 0 and fwd(D=0) == 0 and fwd(T=0, x=None, g=None, y=None) == 0
    # outputs that share bytes with inputs or each other (x: 96 bytes from 1 << 20 on)
    assert fwd(y=at[0]) == 1 and fwd(y=P((1 << 20) + 80)) == 1 and fwd(y=P((1 << 20) - 16)) == 1
    assert fwd(y=at[1]) == 1 and fwd(h=at[0]) == 1 and fwd(m=at[1]) == 1 and fwd(h=at[2]) == 1
    assert fwd(lens=at[3], h=at[3]) == 1 and fwd(m=at[4], h=at[4]) == 1
    assert fwd(h0=at[5], h=P((6 << 20) + 16)) == 1 and fwd(h0=at[5], m=at[5]) == 1

    def bwd(x=at[0], g=at[1], dy=at[2], dt=1, gate=1, lens=None, B=2, T=3, D=4, m=at[3], dh=None,
            dx=at[4], dg=at[5], dh0=None):
        return lib.sanatan_gated_scan_bwd(x, g, dy, dt, gate, lens, B, T, D, m, dh, dx, dg, dh0,
                                          None)

    assert bwd(dt=-1) == 1 and bwd(gate=3) == 1 and bwd(T=-2) == 1
    assert bwd(dy=None) == 1 and bwd(m=None) == 1 and bwd(dx=None) == 1 and bwd(dg=P(8)) == 1
    assert bwd(dh=P(8)) == 1 and bwd(dh0=P(12)) == 1 and bwd(lens=P(24)) == 1
    assert bwd(B=1 << 30, D=2) == 2 and bwd(B=0) == 0
    assert bwd(dx=at[0]) == 1 and bwd(dx=at[5]) == 1 and bwd(dg=at[2]) == 1 and bwd(dg=at[3]) == 1
    assert bwd(dh0=at[4]) == 1 and bwd(dh=at[6], dh0=P((7 << 20) + 16)) == 1
    assert bwd(dh0=at[3]) == 1 and bwd(lens=at[7], dh0=at[7]) == 1

    def step(h=at[0], x=at[1], g=at[2], dt=0, gate=0, N=2, D=4, y=at[3]):
        return lib.sanatan_gated_scan_step(h, x, g, dt, gate, N, D, y, None)

    assert step(h=None) == 1 and step(x=P(2)) == 1 and step(y=None) == 1 and step(N=-1) == 1
    assert step(dt=5) == 1 and step(gate=5) == 1 and step(N=1 << 30, D=4) == 2 and step(N=0) == 0
    assert step(y=at[0]) == 1 and step(y=at[1]) == 1 and step(h=at[2]) == 1 and step(x=at[0]) == 1
    assert lib.sanatan_gated_scan_marks_size(3, 65, 5) == 3 * 2 * 5 * 4
    assert lib.sanatan_gated_scan_marks_size(3, 0, 5) == 0
    assert lib.sanatan_gated_scan_marks_size(-1, 1, 5) == 0


def test_cache_refusals(lib):
    P = ctypes.c_void_p
    ok = P(1 << 20)

    def write(state=ok, z=ok, layers=2, B=3, inner=64, zi=8, pages=ok, n=4, fmt=0, codes=ok,
              scales=ok, zc=ok):
        return lib.sanatan_state_cache_write(state, z, layers, B, inner, zi, pages, n, fmt, codes,
                                             scales, zc, None)

    assert write(fmt=2) == 1 and write(fmt=-1) == 1
    for bad in (dict(layers=-1), dict(B=-1), dict(inner=-1), dict(zi=-1), dict(n=-1)):
        assert write(**bad) == 1, bad
    for bad in (dict(state=None), dict(pages=None), dict(codes=P(8)), dict(scales=P(4)),
                dict(z=None), dict(zc=P(8))):
        assert write(**bad) == 1, bad
    assert write(inner=1 << 41) == 2 and write(inner=1 << 40, B=1 << 20) == 2
    for nothing in (dict(layers=0), dict(B=0), dict(n=0), dict(inner=0, zi=0)):
        assert write(state=None, z=None, pages=None, codes=None, **nothing) == 0, nothing
    assert lib.sanatan_state_cache_read(ok, ok, ok, 4, 7, ok, 1, 1, 64, 0, ok, None, None) == 1
    assert lib.sanatan_state_cache_read(None, ok, ok, 4, 0, ok, 1, 1, 64, 0, ok, None, None) == 1
    assert lib.sanatan_state_cache_read(ok, ok, None, 4, 0, ok, 1, 1, 64, 8, ok, ok, None) == 1


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    from constant_state_recurrence_gb300 import sanatan as S
    x = torch.zeros(1, 2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        S.sanatan_gated_scan_fwd(x, x)
    with pytest.raises(ValueError, match="gate"):
        S._gate("tanh")
    with pytest.raises(ValueError, match="dtype"):
        S.state_cache_empty(1, 64, dtype=torch.float16, device="cpu")
    codes, scales, zc = S.state_cache_empty(3, 70, z_inner=5, layers=2, device="cpu")
    assert codes.shape == (3, 2, 2, 64) and scales.shape == (3, 2, 2) and zc.shape == (3, 2, 5)
    with pytest.raises(ValueError, match="CUDA"):
        S.sanatan_state_cache_write(torch.zeros(2, 1, 70), torch.zeros(1, dtype=torch.int64),
                                    codes, scales, layers=2)
