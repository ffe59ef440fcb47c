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


def test_index_arrays_start_at_any_element(lib):
    for call in (fwd, bwd):     # (B = 0 does nothing, after the optional pointers are looked at)
        assert call(lib, B=0, lens=P(8)) == OK
        assert call(lib, B=0, lens=P(4)) == INVALID
    for call in (write, read):
        assert call(lib, pages=P((2 << 20) + 8)) == UNSUPPORTED
        assert call(lib, pages=P((2 << 20) + 4)) == INVALID


def test_states_start_at_any_element(lib):
    for name in ("h0", "h_out"):
        assert fwd(lib, B=0, **{name: P(4)}) == OK
        assert fwd(lib, B=0, **{name: P(2)}) == INVALID
    for name in ("dh_out", "dh0"):
        assert bwd(lib, B=0, **{name: P(4)}) == OK
        assert bwd(lib, B=0, **{name: P(2)}) == INVALID
    for call in (write, read):
        for name in ("state", "scales", "exact", "exact_cache"):
            args = dict(exact_inner=3, exact=P(5 << 20), exact_cache=P(6 << 20))
            assert call(lib, **{**args, name: P((7 << 20) + 4)}) == UNSUPPORTED, name
            assert call(lib, **{**args, name: P((7 << 20) + 2)}) == INVALID, name
