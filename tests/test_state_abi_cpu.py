"""Host-side argument checks of the gated recurrence and the state cache in the C ABI.
Every call here returns before any device work: nothing is launched."""
import ctypes

import pytest

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED = 0, 1, 2
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    from constant_state_recurrence_gb300 import build, sanatan
    build.build(quiet=True)
    return sanatan.lib()


def fwd(lib, x=P(1 << 20), g=P(2 << 20), dtype=0, gate=0, lens=None, B=1, T=4, D=8, h0=None,
        y=P(3 << 20), h_out=None, marks=None):
    return lib.sanatan_gated_scan_fwd(x, g, dtype, gate, lens, B, T, D, h0, y, h_out, marks, None)


def bwd(lib, x=P(1 << 20), g=P(2 << 20), dy=P(3 << 20), dtype=0, gate=0, lens=None, B=1, T=4,
        D=8, marks=P(4 << 20), dh_out=None, dx=P(5 << 20), dg=P(6 << 20), dh0=None):
    return lib.sanatan_gated_scan_bwd(x, g, dy, dtype, gate, lens, B, T, D, marks, dh_out, dx, dg,
                                      dh0, None)


def write(lib, state=P(1 << 20), exact=None, layers=1, B=1, inner=64, exact_inner=0,
          pages=P(2 << 20), num_pages=BIG, fmt=0, codes=P(3 << 20), scales=P(4 << 20),
          exact_cache=None):
    """(a pool of 2^31 pages is refused after the other checks: UNSUPPORTED stands for
    arguments that are right otherwise)"""
    return lib.sanatan_state_cache_write(state, exact, layers, B, inner, exact_inner, pages,
                                         num_pages, fmt, codes, scales, exact_cache, None)


def read(lib, state=P(1 << 20), exact=None, layers=1, B=1, inner=64, exact_inner=0,
         pages=P(2 << 20), num_pages=BIG, fmt=0, codes=P(3 << 20), scales=P(4 << 20),
         exact_cache=None):
    return lib.sanatan_state_cache_read(codes, scales, exact_cache, num_pages, fmt, pages, layers,
                                        B, inner, exact_inner, state, exact, None)


def test_pages_start_at_any_element(lib):
    for call in (write, read):
        assert call(lib, pages=P((2 << 20) + 8)) == UNSUPPORTED
        assert call(lib, pages=P((2 << 20) + 4)) == INVALID


def test_states_start_at_any_float(lib):
    for call in (write, read):
        for name in ("state", "exact"):
            args = dict(exact_inner=3, exact=P(5 << 20), exact_cache=P(6 << 20))
            assert call(lib, **{**args, name: P((7 << 20) + 4)}) == UNSUPPORTED, name
            assert call(lib, **{**args, name: P((7 << 20) + 2)}) == INVALID, name


def test_scan_refusals(lib):
    for call in (fwd, bwd):
        assert call(lib, dtype=2) == call(lib, gate=2) == call(lib, gate=-1) == INVALID
        assert call(lib, B=-1) == call(lib, T=-1) == call(lib, D=-1) == INVALID
        assert call(lib, B=1 << 16, D=1 << 15) == UNSUPPORTED
        assert call(lib, T=(1 << 30) + 1) == call(lib, D=(1 << 30) + 1) == UNSUPPORTED
        assert call(lib, B=0) == call(lib, D=0) == call(lib, T=0) == OK
        assert call(lib, x=None) == call(lib, g=None) == INVALID
        assert call(lib, x=P((1 << 20) + 4)) == call(lib, g=P((2 << 20) + 8)) == INVALID
    assert fwd(lib, y=None) == fwd(lib, y=P((3 << 20) + 4)) == INVALID
    assert fwd(lib, marks=P((4 << 20) + 4)) == INVALID
    assert fwd(lib, y=P(1 << 20)) == fwd(lib, h_out=P(3 << 20)) == INVALID     # overlaps
    assert fwd(lib, h0=P(7 << 20), h_out=P((7 << 20) + 16)) == INVALID
    for name in ("dy", "marks", "dx", "dg"):
        assert bwd(lib, **{name: None}) == INVALID, name
    assert bwd(lib, dx=P(6 << 20)) == bwd(lib, dg=P(3 << 20)) == INVALID
    assert bwd(lib, dh_out=P(7 << 20), dh0=P((7 << 20) + 16)) == INVALID
    assert lib.sanatan_gated_scan_marks_size(3, 65, 5) == 3 * 2 * 5 * 4
    assert lib.sanatan_gated_scan_marks_size(1, -1, 5) == 0


def test_step_refusals(lib):
    def step(h=P(1 << 20), x=P(2 << 20), g=P(3 << 20), dtype=0, gate=0, N=2, D=8, y=P(4 << 20)):
        return lib.sanatan_gated_scan_step(h, x, g, dtype, gate, N, D, y, None)

    assert step(dtype=5) == step(gate=2) == step(N=-1) == step(D=-2) == INVALID
    assert step(N=1 << 16, D=1 << 15) == UNSUPPORTED and step(N=0) == OK
    for name in "hxgy":
        assert step(**{name: None}) == INVALID
    assert step(y=P(2 << 20)) == step(y=P(1 << 20)) == step(h=P(3 << 20)) == INVALID


def test_cache_refusals(lib):
    for call in (write, read):
        assert call(lib, fmt=2) == call(lib, layers=-1) == call(lib, B=-1) == INVALID
        assert call(lib, inner=-1) == call(lib, exact_inner=-1) == INVALID
        assert call(lib, num_pages=-1) == INVALID
        assert call(lib, layers=0) == call(lib, B=0) == call(lib, inner=0) == OK
        assert call(lib, num_pages=0) == OK
        for name in ("state", "pages", "codes", "scales"):
            assert call(lib, **{name: None}) == INVALID, name
        assert call(lib, exact_inner=1) == INVALID
        assert call(lib, codes=P((3 << 20) + 8)) == INVALID
        n = dict(num_pages=4)
        assert call(lib, inner=(1 << 40) + 1, **n) == UNSUPPORTED
        assert call(lib, layers=1 << 16, B=1 << 15, **n) == UNSUPPORTED
        assert call(lib, inner=1 << 40, B=8, **n) == UNSUPPORTED
        assert call(lib, num_pages=BIG - 1, layers=1 << 10, inner=1 << 20) == UNSUPPORTED
