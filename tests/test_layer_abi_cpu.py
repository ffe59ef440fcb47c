"""Host-side argument checks of the layer norm, the short causal convolution and the
selective scan in the C ABI.  Every call here returns before any device work: nothing is
launched (arguments that are right otherwise are told by a size that is refused last)."""
import ctypes

import pytest

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, NOT_THERE = 0, 1, 2, (3, 4)


def at(n, off=0):
    return P((n << 32) + off)


@pytest.fixture(scope="module")
def lib():
    from constant_state_recurrence_gb300 import build, sanatan
    build.build(quiet=True)
    return sanatan.lib()


def right(status):
    """Past every check: without a GPU the device is asked next, and is not there."""
    import torch
    assert not torch.cuda.is_available(), "these calls are made where nothing can be launched"
    return status in NOT_THERE


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU would run what is past the checks")


def norm_fwd(lib, x=at(1), residual=at(2), weight=at(3), bias=at(4), dtype=0, rows=4, D=8, y=at(5),
             sum=at(6), stats=at(7)):
    return lib.sanatan_layer_norm_fwd(x, residual, weight, bias, dtype, rows, D, 1e-5, y, sum,
                                      stats, None)


def norm_bwd(lib, s=at(1), weight=at(3), dy=at(2), ds=at(4), stats=at(5), dtype=0, rows=4, D=8,
             dx=at(6), dweight=at(7), dbias=at(8), workspace=at(9), ws=1 << 20):
    return lib.sanatan_layer_norm_bwd(s, weight, dy, ds, stats, dtype, rows, D, dx, dweight, dbias,
                                      workspace, ws, None)


def test_norm(lib):
    assert right(norm_fwd(lib)) and right(norm_bwd(lib))
    for call in (norm_fwd, norm_bwd):
        assert call(lib, dtype=2) == call(lib, rows=-1) == call(lib, D=-1) == INVALID
        assert call(lib, rows=1 << 31) == call(lib, D=(1 << 30) + 1) == UNSUPPORTED
        assert call(lib, D=0) == OK
    assert norm_fwd(lib, rows=0) == OK
    for name in ("x", "y"):
        assert norm_fwd(lib, **{name: None}) == norm_fwd(lib, **{name: at(9, 2)}) == INVALID
    for name in ("residual", "weight", "bias", "sum", "stats"):
        assert norm_fwd(lib, **{name: at(9, 2)}) == INVALID, name
    assert right(norm_fwd(lib, residual=None, sum=None, weight=None, bias=None, stats=None))
    assert norm_fwd(lib, residual=None) == INVALID                     # a sum of nothing
    assert right(norm_fwd(lib, dtype=1, x=at(1, 2), y=at(5, 6)))       # any element
    assert norm_fwd(lib, y=at(1)) == norm_fwd(lib, y=at(2, 4)) == norm_fwd(lib, sum=at(1)) == INVALID
    assert right(norm_fwd(lib, sum=at(2))) and norm_fwd(lib, sum=at(2, 4)) == INVALID
    assert norm_fwd(lib, stats=at(5)) == norm_fwd(lib, y=at(6)) == INVALID
    for name in ("s", "dy", "stats", "dx", "workspace"):
        assert norm_bwd(lib, **{name: None}) == INVALID, name
    for name in ("s", "dy", "ds", "dx", "weight", "dweight", "dbias", "workspace"):
        assert norm_bwd(lib, **{name: at(12, 2)}) == INVALID, name
    assert norm_bwd(lib, dx=at(1)) == norm_bwd(lib, dx=at(2)) == norm_bwd(lib, dweight=at(8)) == INVALID
    need = lib.sanatan_layer_norm_bwd_workspace_size(4, 8)
    assert need > 0 and norm_bwd(lib, ws=need - 1) == INVALID and right(norm_bwd(lib, ws=need))
    assert right(norm_bwd(lib, dweight=None, dbias=None, workspace=None, ws=0))
    assert lib.sanatan_layer_norm_bwd_workspace_size(0, 8) == 0


def conv_fwd(lib, x=at(1), ldx=8, w=at(2), bias=at(3), dtype=0, act=1, lens=at(4), B=2, T=5, D=8,
             K=4, s0=at(5), y=at(6), s_out=at(7)):
    return lib.sanatan_causal_conv_fwd(x, ldx, w, bias, dtype, act, lens, B, T, D, K, s0, y, s_out,
                                       None)


def conv_bwd(lib, x=at(1), ldx=8, w=at(2), bias=at(3), dy=at(4), dtype=0, act=1, lens=at(5), B=2,
             T=5, D=8, K=4, s0=at(6), ds_out=at(7), dx=at(8), dw=at(9), dbias=at(10), ds0=at(11),
             workspace=at(12), ws=1 << 20):
    return lib.sanatan_causal_conv_bwd(x, ldx, w, bias, dy, dtype, act, lens, B, T, D, K, s0,
                                       ds_out, dx, dw, dbias, ds0, workspace, ws, None)


def conv_step(lib, state=at(1), x=at(2), ldx=8, w=at(3), bias=at(4), dtype=0, act=0, N=3, D=8, K=4,
              y=at(5)):
    return lib.sanatan_causal_conv_step(state, x, ldx, w, bias, dtype, act, N, D, K, y, None)


def test_conv(lib):
    assert right(conv_fwd(lib)) and right(conv_bwd(lib)) and right(conv_step(lib))
    for call in (conv_fwd, conv_bwd, conv_step):
        assert call(lib, dtype=-1) == call(lib, act=2) == call(lib, K=0) == call(lib, D=-1) == INVALID
        assert call(lib, ldx=7) == call(lib, x=None) == call(lib, w=None) == INVALID
        assert call(lib, K=9) == call(lib, D=(1 << 30) + 1, ldx=1 << 40) == UNSUPPORTED
        assert call(lib, D=0) == OK
        assert call(lib, w=at(15, 2)) == call(lib, bias=at(15, 1)) == call(lib, x=at(15, 2)) == INVALID
        assert right(call(lib, x=at(15, 4), bias=None))
    for call in (conv_fwd, conv_bwd):
        assert call(lib, B=-1) == call(lib, T=-1) == INVALID
        assert call(lib, B=1 << 16, D=1 << 15, ldx=1 << 15) == UNSUPPORTED
        assert call(lib, T=(1 << 30) + 1) == call(lib, ldx=1 << 58) == UNSUPPORTED
        assert call(lib, B=1 << 15, T=1 << 29, D=1 << 15, ldx=1 << 15) == UNSUPPORTED
        assert call(lib, lens=at(15, 4)) == call(lib, s0=at(15, 2)) == INVALID
        assert right(call(lib, lens=None, s0=None)) and right(call(lib, lens=at(15, 8)))
    assert conv_fwd(lib, B=0) == OK
    assert conv_fwd(lib, y=None) == conv_fwd(lib, y=at(1)) == conv_fwd(lib, s_out=at(5)) == INVALID
    assert conv_fwd(lib, y=at(1, 4 * 8 * 5 * 2 - 4)) == INVALID             # the last value
    assert conv_fwd(lib, ldx=16, y=at(1, 4 * (16 * 9 + 8) - 4)) == INVALID  # of wide rows
    assert right(conv_fwd(lib, ldx=16, y=at(1, 4 * (16 * 9 + 8))))
    for name in ("dy", "dx", "workspace"):
        assert conv_bwd(lib, **{name: None}) == INVALID, name
    for name in ("dy", "dx", "ds_out", "dw", "dbias", "ds0", "workspace"):
        assert conv_bwd(lib, **{name: at(15, 2)}) == INVALID, name
    for name, other in (("dx", 1), ("dx", 4), ("dw", 2), ("ds0", 7), ("dw", 10), ("ds0", 12)):
        assert conv_bwd(lib, **{name: at(other)}) == INVALID, name
    need = lib.sanatan_causal_conv_bwd_workspace_size(2, 5, 8, 4)
    assert need > 0 and conv_bwd(lib, ws=need - 1) == INVALID and right(conv_bwd(lib, ws=need))
    assert right(conv_bwd(lib, dw=None, dbias=None, workspace=None, ws=0))
    assert conv_step(lib, N=-1) == conv_step(lib, state=None) == conv_step(lib, y=at(2)) == INVALID
    assert conv_step(lib, N=0) == OK and right(conv_step(lib, K=1, state=None))


def scan_fwd(lib, u=at(1), dt=at(2), z=at(3), ldz=8, Bm=at(4), ldb=16, Cm=at(5), ldc=16, A=at(6),
             skip=at(7), dt_bias=at(8), dtype=0, softplus=1, lens=at(9), B=2, T=5, D=8, N=16,
             h0=at(10), y=at(11), h_out=at(12), marks=at(13), workspace=None, ws=0):
    return lib.sanatan_selective_scan_fwd(u, dt, z, ldz, Bm, ldb, Cm, ldc, A, skip, dt_bias, dtype,
                                          softplus, lens, B, T, D, N, h0, y, h_out, marks,
                                          workspace, ws, None)


def scan_bwd(lib, u=at(1), dt=at(2), z=at(3), ldz=8, Bm=at(4), ldb=16, Cm=at(5), ldc=16, A=at(6),
             skip=at(7), dt_bias=at(8), dtype=0, softplus=1, lens=at(9), B=2, T=5, D=8, N=16,
             dy=at(10), marks=at(11), dh_out=at(12), du=at(13), ddt=at(14), dz=at(15), dA=at(16),
             dB=at(17), dC=at(18), dskip=at(19), ddt_bias=at(20), dh0=at(21), workspace=at(22),
             ws=1 << 24):
    return lib.sanatan_selective_scan_bwd(u, dt, z, ldz, Bm, ldb, Cm, ldc, A, skip, dt_bias, dtype,
                                          softplus, lens, B, T, D, N, dy, marks, dh_out, du, ddt,
                                          dz, dA, dB, dC, dskip, ddt_bias, dh0, workspace, ws,
                                          None)


def scan_step(lib, h=at(9), u=at(1), dt=at(2), z=at(3), ldz=8, Bm=at(4), ldb=16, Cm=at(5), ldc=16,
              A=at(6), skip=at(7), dt_bias=at(8), dtype=0, softplus=1, nseq=3, D=8, N=16, y=at(10)):
    return lib.sanatan_selective_scan_step(h, u, dt, z, ldz, Bm, ldb, Cm, ldc, A, skip, dt_bias,
                                           dtype, softplus, nseq, D, N, y, None)


def test_scan(lib):
    assert right(scan_fwd(lib)) and right(scan_bwd(lib)) and right(scan_step(lib))
    for call in (scan_fwd, scan_bwd, scan_step):
        assert call(lib, dtype=2) == call(lib, D=-1) == call(lib, N=0) == INVALID
        assert call(lib, ldb=15) == call(lib, ldc=15) == call(lib, ldz=7) == INVALID
        assert call(lib, N=129, ldb=129, ldc=129) == UNSUPPORTED
        assert call(lib, D=(1 << 30) + 1, ldz=1 << 40) == UNSUPPORTED
        for name in ("u", "dt", "Bm", "Cm", "A"):
            assert call(lib, **{name: None}) == call(lib, **{name: at(30, 2)}) == INVALID, name
        for name in ("z", "skip", "dt_bias"):
            assert call(lib, **{name: at(30, 2)}) == INVALID, name
        assert right(call(lib, skip=None, dt_bias=None))
        assert right(call(lib, u=at(30, 4), Bm=at(31, 12), A=at(32, 4)))
    assert scan_fwd(lib, D=0) == scan_step(lib, D=0) == OK
    # without channels dB and dC are still there, and zeros
    none = dict(D=0, u=None, dt=None, z=None, A=None, dy=None, marks=None, du=None, ddt=None,
                dz=None, dA=None, workspace=None, ws=0)
    assert right(scan_bwd(lib, **none))
    assert scan_bwd(lib, **none, T=0) == scan_bwd(lib, **none, B=0) == OK
    for name in ("dB", "dC"):
        for wrong in (None, at(30, 2), at(4), at(5)):
            assert scan_bwd(lib, **dict(none, **{name: wrong})) == INVALID, name
    for call in (scan_fwd, scan_bwd):
        assert call(lib, B=-1) == call(lib, T=-1) == INVALID
        assert call(lib, B=1 << 16, D=1 << 15, ldz=1 << 15) == UNSUPPORTED
        assert call(lib, T=(1 << 30) + 1) == call(lib, ldb=1 << 58) == UNSUPPORTED
        assert call(lib, lens=at(30, 4)) == INVALID and right(call(lib, lens=None))
    assert scan_fwd(lib, B=0) == OK and scan_fwd(lib, T=0, h_out=None) == OK
    assert scan_fwd(lib, y=None) == scan_fwd(lib, h0=at(30, 2)) == scan_fwd(lib, marks=at(30, 2)) == INVALID
    for other in range(1, 14):
        if other != 11:
            assert scan_fwd(lib, y=at(other)) == INVALID, other
    assert right(scan_fwd(lib, h_out=at(10))) and scan_fwd(lib, h_out=at(10, 4)) == INVALID
    assert right(scan_fwd(lib, z=None, ldz=0))
    need = lib.sanatan_selective_scan_fwd_workspace_size(1, 4096, 8, 16)
    big = dict(B=1, T=4096)
    assert need > 0 and scan_fwd(lib, **big) == INVALID
    assert scan_fwd(lib, **big, workspace=at(30), ws=need - 1) == INVALID
    assert right(scan_fwd(lib, **big, workspace=at(30), ws=need))
    assert scan_fwd(lib, **big, workspace=at(1), ws=need) == INVALID
    for name in ("dy", "marks", "du", "ddt", "dz", "dA", "dB", "dC", "workspace"):
        assert scan_bwd(lib, **{name: None}) == INVALID, name
    assert scan_bwd(lib, z=None) == INVALID and right(scan_bwd(lib, z=None, dz=None, ldz=0))
    for name, other in (("du", 1), ("ddt", 2), ("dz", 3), ("dB", 4), ("dC", 5), ("dA", 6),
                        ("dskip", 7), ("ddt_bias", 8), ("du", 10), ("dA", 11), ("dh0", 11),
                        ("du", 14), ("dB", 18), ("workspace", 13)):
        assert scan_bwd(lib, **{name: at(other)}) == INVALID, (name, other)
    assert right(scan_bwd(lib, dh0=at(12))) and scan_bwd(lib, dh0=at(12, 4)) == INVALID
    need = lib.sanatan_selective_scan_bwd_workspace_size(2, 5, 8, 16)
    assert scan_bwd(lib, ws=need - 1) == INVALID and right(scan_bwd(lib, ws=need))
    assert right(scan_bwd(lib, dskip=None, ddt_bias=None, dh0=None, dh_out=None))
    assert scan_step(lib, nseq=-1) == scan_step(lib, h=None) == scan_step(lib, y=None) == INVALID
    assert scan_step(lib, y=at(9)) == scan_step(lib, h=at(1)) == INVALID and scan_step(lib, nseq=0) == OK
    assert lib.sanatan_selective_scan_marks_size(2, 17, 8, 16) == 2 * 2 * 8 * 16 * 4
    assert lib.sanatan_selective_scan_marks_size(2, -1, 8, 16) == 0


def test_sizes_that_are_not_asked_for(lib):
    for args in ((-1, 5, 8, 16), (2, -5, 8, 16), (2, 5, -8, 16), (2, 5, 8, 0), (2, 5, 8, 129)):
        assert lib.sanatan_selective_scan_fwd_workspace_size(*args) == 0
        assert lib.sanatan_selective_scan_bwd_workspace_size(*args) == 0
    assert lib.sanatan_causal_conv_bwd_workspace_size(0, 5, 8, 4) == 0
