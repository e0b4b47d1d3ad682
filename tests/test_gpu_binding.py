"""The two ways through the Python binding of the step calls: that the short one gives and takes what the other does, and that
nothing but its speed depends on it."""
import threading
import time
import warnings

import pytest
import torch

from gpu_util import DEV, built
from test_gpu_step import BF, Case, i32
from w6a8_quantized_linear_gb300 import build, qlin

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


def calls():
    """Each call that has a short way, with fresh outputs; what it gave."""
    c = Case([40, 9], 2, 2, 64, 16, BF, seed=2, parents=[-1, 0])
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(4, h * 64, generator=g).to(DEV) for h in (4, 2, 2))
    q_out = torch.empty(4, 4 * 64, dtype=BF, device=DEV)
    qlin.kv_append(c.cache, c.step, q, k, v, turns=qlin.rope_turns(1e4, 64, device=DEV), q_out=q_out)
    stats = torch.empty(4, 4, 2, device=DEV)
    qlin.tree_attention(c.cache, c.step, q_out, stats=stats)
    score = torch.zeros(2, 2, 50, device=DEV)
    qlin.kv_weigh(c.cache, c.step, q_out, stats, score)
    weighed = score.clone()
    ws = qlin.new_workspace(qlin.kv_evict_workspace_bytes(c.cache, c.step, 50), DEV)
    qlin.kv_evict(c.cache, c.step, score, i32([20, 5]), len_out=c.step.len, ws=ws)
    logits = torch.randn(3, 1000, generator=g).to(DEV)
    adjusted = qlin.adjust_logits(logits, out=torch.empty_like(logits), history=i32([[5, 6]] * 3), frequency=torch.ones(3, device=DEV))
    return q_out, weighed, score[:, :, :5], c.step.len, adjusted


@pytest.mark.parametrize("fault", ["missing", "no library", "another torch's"])
def test_without_the_extension_calls_go_the_other_way(fault, monkeypatch, tmp_path):
    """... with a warning, once, and the same results."""
    want = calls()
    monkeypatch.setattr(qlin, "_binding", None)
    broken = tmp_path / "_qlin_binding.so"
    if fault == "no library":
        broken.write_bytes(b"none")
        monkeypatch.setattr(build, "binding_fits", lambda: True)
    elif fault == "another torch's":
        monkeypatch.setattr(torch, "__version__", "1.0")
    if fault != "another torch's":
        monkeypatch.setattr(build, "BINDING", str(broken))
    with pytest.warns(RuntimeWarning, match="_qlin_binding"):
        got = calls()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        calls()


def test_pairs_is_any_truth_value():
    c = Case([7], 3, 2, 64, 16, BF, seed=2, fill=False)
    q = torch.randn(3, 4 * 64, generator=torch.Generator().manual_seed(3)).to(DEV)
    turns, out = qlin.rope_turns(1e4, 64, device=DEV), [torch.empty(3, 4 * 64, dtype=BF, device=DEV) for _ in range(3)]
    for o, pairs in zip(out, (True, 2, "yes")):
        qlin.kv_append(c.cache, c.step, q, turns=turns, pairs=pairs, q_out=o)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
