"""Sequences cut into segments for every count of lanes that is cut (4, 8 and 16 of four
states), at rows of words and at rows that start anywhere, both types, against the float64
definitions and bounds of test_gpu_selective_scan."""
import pytest
import torch

from constant_state_recurrence_gb300 import sanatan as S
from test_gpu_layer_norm import BF16, F32
from test_gpu_selective_scan import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,T,D,N,lens", [
    (1, 160, 16, 16, None), (2, 140, 24, 16, [140, 3]),                    # four lanes
    (1, 150, 5, 20, None), (2, 131, 16, 32, [94, 131]), (1, 200, 24, 24, [70]),   # eight
    (1, 260, 40, 32, [0]), (1, 140, 17, 31, None),
    (1, 150, 8, 64, None), (2, 135, 16, 64, [135, 60]), (1, 200, 9, 48, [10]),    # sixteen
    (1, 300, 16, 40, [299]), (1, 140, 3, 33, None)])
def test_segments_of_every_lane_count(b, T, D, N, lens, dtype):
    """Lengths that end in the last segment, before it, in the first and at no token."""
    assert S.selective_scan_fwd_workspace_size(b, T, D, N) > 0
    check(b, T, D, N, dtype, seed=T + N, h0=T % 20 != 0, gated=D % 3 != 0, lens=lens)


@pytest.mark.parametrize("N", [16, 32, 64])
def test_segments_of_parts_of_larger_tensors(N):
    def place(t):
        big = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda:0")
        big[1:].copy_(t.flatten())
        return big[1:].view(t.shape)
    check(1, 140, 16, N, BF16, place=place, seed=N)
