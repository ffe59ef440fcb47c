"""The selective scan's backward keeps dB's and dC's parts, one for every block of channels,
within 512 MB or the marks that the forward left, whichever is more.  Sizes alone, on the CPU."""
import pytest

from constant_state_recurrence_gb300 import sanatan as S


@pytest.fixture(scope="module", autouse=True)
def built():
    from constant_state_recurrence_gb300 import build
    build.build(quiet=True)


@pytest.mark.parametrize("b,T,D,N", [
    (4, 4096, 4096, 128), (8, 4096, 1536, 128), (8, 4096, 1536, 64), (8, 4096, 1536, 32),
    (1, 32768, 1536, 64), (2, 4096, 2048, 64), (1, 16384, 8192, 100), (64, 100000, 512, 128),
    (8, 4096, 1536, 16), (8, 4096, 8192, 16), (300, 60, 4096, 128), (1, 1 << 20, 64, 128)])
def test_the_backwards_workspace(b, T, D, N):
    """Parts, with up to a third for the last piece's share; beside them five copies of the
    state for each segment at most (a part of dA, the gradient carried, sums over tokens),
    and no more segments than make six blocks an SM, of four tiles of sixteen tokens."""
    marks = int(S.lib().sanatan_selective_scan_marks_size(b, T, D, N))
    size = S.selective_scan_bwd_workspace_size(b, T, D, N)
    segments = max(1, min(-(-6 * 152 * 32 // (b * D)) + 1, T // 64))
    assert 0 < size <= 4 / 3 * max(1 << 29, marks) + 5 * 4 * b * D * N * segments
