"""Layer calls of host threads at once, each on a stream of its own, give what they give alone."""
import threading

import pytest
import torch

from constant_state_recurrence_gb300 import sanatan as S
from gpu_util import dev
from test_gpu_layer_norm import BF16, F32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,widths", [(F32, (2048, 4096)), (F32, (768, 1024)),
                                          (BF16, (2560, 8192)), (F32, (771, 4095))])
def test_norm_backwards_of_different_widths(dtype, widths):
    """The blocks of the widths take different amounts of shared memory of one kernel."""
    work = []
    for D in widths:
        x, _, dy, ds, w, b = (t.to(dev()) for t in make(200, D, dtype, D))
        _, _, stats = S.sanatan_layer_norm_fwd(x, w, b, want_stats=True)
        work.append((x, w, dy, stats, ds))
    want = [S.sanatan_layer_norm_bwd(*a) for a in work]
    torch.cuda.synchronize()
    gate, wrong = threading.Barrier(len(work)), []

    def run(a, ref):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                for _ in range(300):
                    got = S.sanatan_layer_norm_bwd(*a)
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(got[k], ref[k]) for k in ref):
                wrong.append("other values")
        except Exception as e:   # (the thread's own: told below)
            wrong.append(repr(e))
    threads = [threading.Thread(target=run, args=p) for p in zip(work, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
