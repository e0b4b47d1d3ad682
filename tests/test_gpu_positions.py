"""Appending at given positions of several axes on the GPU against a plain 64-bit form."""
import math

import pytest
import torch

import step_ref as R
from gpu_util import DEV, built
from test_gpu_step import BF, FP, Case, i32
from w6a8_quantized_linear_gb300 import qlin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built()
    torch.cuda.set_device(DEV)


def turned(x, gamma, position, axis, radians, pairs):
    """x [H, D]: each pair's angle is its axis' position times its frequency."""
    return R.append_row(x, gamma, 1e-6, 1, [position[a] * f for a, f in zip(axis, radians)], pairs)


CASES = [
    # lens, T, Hq, heads, width, page, dtype, src, sections, dealt, pairs, layout
    ([0], 1, 4, 4, 64, 16, BF, torch.float32, (12, 10, 10), True, False, "hnd"),
    ([15], 1, 24, 4, 256, 64, BF, torch.float32, (12, 10, 10), True, False, "hnd"),
    ([100, 3, 16], 8, 12, 2, 128, 16, FP, torch.float32, (24, 20, 20), False, True, "nhd"),
    ([40], 67, 6, 1, 256, 128, BF, torch.bfloat16, (32, 32, 64), True, False, "hnd"),
    ([7, 250], 33, 6, 3, 64, 32, FP, torch.bfloat16, (1, 0, 2, 5), True, True, "pool"),
    ([31], 5, 3, 3, 128, 16, BF, torch.float32, (0, 7), False, False, "hnd"),
    ([9], 3, 2, 1, 64, 16, FP, torch.bfloat16, (32,), False, False, "hnd"),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_append_at_positions_against_64_bits(case):
    lens, T, Hq, heads, D, page, dtype, src, sections, dealt, pairs, layout = case
    c = Case(lens, T, heads, D, page, dtype, layout, seed=3, fill=False, tree="none")
    g = torch.Generator().manual_seed(12)
    n, axes = len(lens) * T, len(sections)
    q = (torch.randn(n, Hq * D, generator=g) * 3).to(src)
    k = (torch.randn(n, heads * D, generator=g) * 0.2).to(src)
    v = torch.randn(n, heads * D, generator=g).to(src)
    qg, kg = 0.5 + torch.rand(D, generator=g), 0.5 + torch.rand(D, generator=g)
    position = torch.randint(-300, 1 << 20, (n, axes), generator=g, dtype=torch.int32)
    axis = qlin.rope_axes(sections, dealt)
    rot = 2 * len(axis)
    radians = [1e6 ** (-2.0 * i / rot) for i in range(rot // 2)]
    wide = torch.full((n, axes + 3), -1, dtype=torch.int32)  # rows of a wider tensor
    wide[:, :axes] = position
    out = qlin.kv_append(c.cache, c.step, q=q.to(DEV), k=k.to(DEV), v=v.to(DEV), q_gamma=qg.to(DEV), k_gamma=kg.to(DEV),
                         turns=qlin.rope_turns(1e6, rot, device=DEV), pairs=pairs, position=wide.to(DEV)[:, :axes], axis=axis)
    out = out.cpu().double().view(n, Hq, D)
    for b in range(len(lens)):
        gk, gv = c.get(b, lens[b], T)
        for t in range(T):
            row = b * T + t
            at = position[row].tolist()
            for got, x, gamma, H in ((out[row], q, qg, Hq), (gk[t].double(), k, kg, heads)):
                want = turned(x[row].view(H, D), gamma, at, axis, radians, pairs)
                assert ((got - want).abs() <= R.append_bound(want, dtype)).all()
            assert torch.equal(gv[t], v[row].view(heads, D).to(dtype))


def test_one_axis_of_the_same_positions_changes_nothing():
    """len + depth given as positions: the same bits, counts and absent sequences left alone."""
    T, D = 9, 128
    g = torch.Generator().manual_seed(4)
    rows = [torch.randn(3 * T, h * D, generator=g).to(DEV) for h in (6, 2, 2)]
    turns = qlin.rope_turns(1e4, D, device=DEV)
    got = []
    for given in (False, True):
        c = Case([20, -1, 5], T, 2, D, 16, BF, seed=1, fill=False, tree="none", count=[T, T, 4])
        at = i32([max(n, 0) + t for n in (20, -1, 5) for t in range(T)])
        out = torch.full((3 * T, 6 * D), 7.0, dtype=BF, device=DEV)
        qlin.kv_append(c.cache, c.step, *rows, turns=turns, q_out=out, position=at if given else None)
        got.append((out, c.k.nan_to_num(nan=9.0), c.v.nan_to_num(nan=9.0)))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_positions_are_read_at_replay():
    c = Case([3], 2, 1, 64, 16, FP, seed=2, fill=False, tree="none")
    q = torch.randn(2, 64, generator=torch.Generator().manual_seed(1)).to(DEV)
    at, turns = i32([[0, 0], [0, 0]]), qlin.rope_turns(1e4, 64, device=DEV)
    axis = qlin.rope_axes((16, 16), dealt=True)
    out = torch.empty(2, 64, dtype=FP, device=DEV)
    call = lambda: qlin.kv_append(c.cache, c.step, q=q, turns=turns, q_out=out, position=at, axis=axis)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    at.copy_(i32([[5, 1000], [-3, 2]]))
    graph.replay()
    radians = [1e4 ** (-2.0 * i / 64) for i in range(32)]
    for t, p in enumerate(([5, 1000], [-3, 2])):
        want = turned(q[t].cpu().view(1, 64), None, p, axis, radians, False)
        assert ((out[t].cpu().double() - want[0]).abs() <= R.append_bound(want, FP)[0]).all()
        assert math.isfinite(float(out.float().sum()))
