"""The selective scan with steps of both signs and decays above one (softplus=False), against
the float64 definitions.

The bounds are those of test_gpu_selective_scan.  A path p_t = A sum delta that goes up and
down lets what was put into a state at its lowest grow by exp(range); inputs and gradients are
scaled by 1e-15, so that no value leaves float32 where the definition's do not, while the
products of a tile's decays alone do.  Segments: the sum of a segment's steps has a rounding
for each of its tiles and four more, of at most e times the sum of |delta|.  Its share of
an exponent, (tiles + 4) e sum |delta A|, is what the bounds allow the decays of the same tokens,
(16 tokens + 6 sum |delta A|) e, where tiles - 2 times the average |delta A| is at most 16: here
segments have five tiles, one in three of them with steps of 15 on average."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as R
from constant_state_recurrence_gb300 import sanatan as S
from gpu_util import dev, f64
from test_gpu_layer_norm import BF16, F32, close
from test_gpu_selective_scan import bounds, make, on

pytestmark = pytest.mark.gpu

SMALL = 1e-15


def against(x, dy, dh, dtype, lens=None):
    """Forward's and backward's outputs within their bounds."""
    d = on(x)
    h0 = d.pop("h0")
    ln = None if lens is None else torch.tensor(lens).to(dev())
    y, h, marks = S.sanatan_selective_scan_fwd(**d, softplus=False, h0=h0, lens=ln,
                                               want_state=True, want_marks=True)
    g = S.sanatan_selective_scan_bwd(**d, dy=dy.to(dev()), marks=marks, softplus=False, lens=ln,
                                     dh_last=None if dh is None else dh.to(dev()), want_dh0=True)
    n = {k: None if t is None else f64(t) for k, t in x.items()}
    b, T = n["u"].shape[:2]
    cut = None if lens is None else R.lengths(lens, b, T)
    args = dict(n, soft=False, lens=cut)
    y_ref, h_ref, before = R.selective_scan(**args)
    ref = R.selective_scan_backward(**args, dy=f64(dy), dh_last=None if dh is None else f64(dh))
    bd = bounds(n, False, cut, f64(dy), None if dh is None else f64(dh))
    real = np.ones((b, T), bool) if cut is None else np.arange(T)[None] < np.asarray(cut)[:, None]
    close(y, y_ref, bd["y"] * real[..., None] + 1e-34, dtype, "y")
    close(h, h_ref, bd["last"] + 1e-34, F32, "h_last")
    real = real[:, ::16]
    close(marks[torch.from_numpy(real).to(dev())], before[:, ::16][real], bd["marks"][real] + 1e-34,
          F32, "marks")
    for k in ("du", "ddt", "dz", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"):
        if g[k] is not None:
            close(g[k], ref[k], bd[k] + 1e-34, dtype if k in ("du", "ddt", "dz", "dB", "dC") else F32,
                  k)


def up_and_down(b, T, D, N, dtype, seed, gated, every=1, far=False):
    """Steps whose sums wander between -50 and 50, by at most 40 a step, and every sixteen tokens
    come back to where they were but for one (of every-th tiles; the others' steps are up to
    0.2); the last third of the channels has only such small steps of both signs.  far: the
    sums go up to 90 away from where a tile begins, to one side."""
    x, dy, dh = make(b, T, D, N, dtype, seed, gated, h0=True)
    rng = np.random.default_rng(seed)
    dt, p = np.zeros((b, T, D)), np.zeros((b, D))
    home = np.zeros((b, D))
    for t in range(T):
        if t // 16 % every:
            continue
        if t % 16 == 0:
            home = p
        lo, hi = (-5, 90) if far else (-50, 50)
        aim = np.where(np.arange(D) % 2 > 0, 1, -1) * rng.uniform(lo, hi, (b, D)) if t % 16 < 13 else home + rng.uniform(-1, 1, (b, D))
        step = torch.from_numpy(np.clip(aim - p, -40, 40)).to(dtype).double().numpy()
        dt[:, t], p = step, p + step
    calm = (np.arange(T)[:, None] // 16 % every > 0) | (np.arange(D) >= D - D // 3)
    dt = np.where(calm, rng.uniform(-0.2, 0.2, (b, T, D)), dt)
    x["dt"], x["dt_bias"] = torch.from_numpy(dt).to(dtype), None
    size = 0.3 + 0.7 * torch.rand(D, N, generator=torch.Generator().manual_seed(seed))
    x["A"] = size * torch.where(torch.arange(N) % 3 == 1, 1.0, -1.0)
    for k in ("u", "h0"):
        x[k] = x[k] * SMALL
    return x, dy * SMALL, dh * SMALL


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,T,D,N", [(2, 50, 33, 16), (3, 90, 40, 16), (1, 67, 8, 32),
                                     (1, 40, 7, 50), (1, 35, 4, 128)])
def test_steps_of_both_signs(b, T, D, N, dtype, far):
    x, dy, dh = up_and_down(b, T, D, N, dtype, T + N, gated=D % 2 == 0, far=far)
    against(x, dy, dh, dtype)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,T,D,N", [(1, 300, 24, 16), (2, 200, 9, 7), (1, 150, 8, 64)])
def test_steps_of_both_signs_in_segments(b, T, D, N, dtype, far):
    assert S.selective_scan_fwd_workspace_size(b, T, D, N) > 0
    x, dy, dh = up_and_down(b, T, D, N, dtype, T + N, gated=D % 2 == 0, every=3, far=far)
    against(x, dy, dh, dtype, lens=[T - 21, T][:b])


@pytest.mark.parametrize("A,steps", [(-16.0, (-3, -3, 3, 3)), (-1.0, (-50, -50, 50, 50)),
                                     (2.0, (30, 30, -30, -30))])
def test_a_tile_whose_decays_leave_float32(A, steps):
    """Four steps, then none: the state stays what the last step left, the step itself to e^-48,
    and is what single tokens leave.  (The first three inputs cancel to a rounding of the third,
    which the last decay takes away: 8 e are the last token's own.)"""
    T, D, N = 40, 32, 16
    dt = torch.zeros(1, T, D)
    dt[0, :4] = torch.tensor(steps, dtype=F32)[:, None]
    one = torch.ones(1, T, N)
    d = [t.to(dev()) for t in (torch.ones(1, T, D), dt, torch.full((D, N), A), one, one)]
    y, h, _ = S.sanatan_selective_scan_fwd(*d, softplus=False, want_state=True)
    h1, h64 = torch.zeros(1, D, N, device=dev()), 0.0
    for t in range(T):
        y1 = S.sanatan_selective_scan_step(h1, *(p[:, t].contiguous() for p in d[:2]), d[2],
                                           *(p[:, t].contiguous() for p in d[3:]), softplus=False)
        step = float(dt[0, t, 0])
        h64 = np.exp(step * A) * h64 + step
        if t >= 4:
            assert torch.equal(y[:, t], y[:, 4])
    assert abs(h64) > 1
    room = 8 * 2.0 ** -24
    assert np.abs(f64(h) / h64 - 1).max() <= room
    assert np.abs(f64(h1) / h64 - 1).max() <= room
    assert np.abs(f64(y1) / (N * h64) - 1).max() <= room + 8 * 2.0 ** -24


@pytest.mark.parametrize("D,N", [(8, 16), (5, 7), (8, 40)])
def test_segments_of_growing_states(D, N):
    """A segment's decay may be beyond float32 where no state is: nothing put in before the
    last tokens, and gradients of the first alone."""
    x, dy, _ = make(1, 256, D, N, F32, D + N, gated=False, h0=False)
    x["A"], x["dt"], x["dt_bias"] = x["A"].abs().clamp(1.5, 2.0), torch.ones(1, 256, D), None
    assert S.selective_scan_fwd_workspace_size(1, 256, D, N) > 0
    x["u"][:, :-25] = 0
    dy[:, 25:] = 0
    against(x, dy, None, F32)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D,N", [(8, 16), (3, 33)])
def test_a_segment_carries_what_fits(D, N, sign):
    """Two segments: exp(102) up and as much down, or down and up.  A state that has the room
    for it is carried, though the segment's decay alone has none in float32.  (No inputs: the
    state is a product of 128 decays, each off by 20 e, and of the segments' exponents, which
    are exact but for the power of two: 3000 e.)"""
    T = 128
    dt = torch.ones(1, T, D) * sign
    dt[:, T // 2:] = -sign
    A = torch.full((D, N), 1.6)
    h0 = (1 + torch.rand(1, D, N, generator=torch.Generator().manual_seed(1))) * \
        (1e-30 if sign > 0 else 1e20)
    assert S.selective_scan_fwd_workspace_size(1, T, D, N) > 0
    zero, one = torch.zeros(1, T, D), torch.ones(1, T, N)
    d = [t.to(dev()) for t in (zero, dt, A, one, one)]
    y, h, marks = S.sanatan_selective_scan_fwd(*d, softplus=False, h0=h0.to(dev()),
                                               want_state=True, want_marks=True)
    path = np.cumsum(f64(dt)[0, :, 0] * np.float64(np.float32(1.6)))
    assert np.abs(f64(h) / (f64(h0) * np.exp(path[-1])) - 1).max() <= 3000 * 2.0 ** -24
    want = (f64(h0)[0].sum(-1) * np.exp(path)[:, None])
    assert np.abs(f64(y)[0] / want - 1).max() <= 3000 * 2.0 ** -24
    dh = torch.full((1, D, N), 1e20 if sign > 0 else 1e-30)    # (from behind: the other way)
    g = S.sanatan_selective_scan_bwd(*d, zero.to(dev()), marks, softplus=False,
                                     dh_last=dh.to(dev()), want_dh0=True)
    assert np.abs(f64(g["dh0"]) / (f64(dh) * np.exp(path[-1])) - 1).max() <= 3000 * 2.0 ** -24
