"""The two ways through the Python binding of the step calls: that the short one gives and takes what the other does, and that
nothing but its speed depends on it."""
import threading
import time

import pytest
import torch

from gpu_util import DEV, built
from test_gpu_step import BF, Case
from w6a8_quantized_linear_gb300 import qlin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built()
    torch.cuda.set_device(DEV)


def test_other_threads_run_while_a_launch_waits():
    """A stream's queue of launches is full behind a kernel of most of a second: who launches into it waits, no other thread."""
    x = torch.randn(1, 64, device=DEV)
    out = torch.empty_like(x)
    qlin.adjust_logits(x, out=out)
    torch.cuda.synchronize()
    took = []

    def launch():
        t = time.perf_counter()
        for _ in range(4000):  # more than a queue holds
            qlin.adjust_logits(x, out=out)
        took.append(time.perf_counter() - t)

    thread = threading.Thread(target=launch)
    torch.cuda._sleep(1_500_000_000)
    last, gap = time.perf_counter(), 0.0
    thread.start()
    while thread.is_alive():
        time.sleep(1e-3)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    thread.join()
    torch.cuda.synchronize()
    assert took[0] > 0.4 and gap < 0.2, (took, gap)


def test_pairs_is_any_truth_value():
    c = Case([7], 3, 2, 64, 16, BF, seed=2, fill=False)
    q = torch.randn(3, 4 * 64, generator=torch.Generator().manual_seed(3)).to(DEV)
    turns, out = qlin.rope_turns(1e4, 64, device=DEV), [torch.empty(3, 4 * 64, dtype=BF, device=DEV) for _ in range(3)]
    for o, pairs in zip(out, (True, 2, "yes")):
        qlin.kv_append(c.cache, c.step, q, turns=turns, pairs=pairs, q_out=o)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
