"""Eviction by accumulated weight on the GPU against its definition: what stays, what moves where, and what is left alone."""
import math

import numpy as np
import pytest
import torch

from gpu_util import DEV, built
from test_gpu_step import BF, FP, Case, i32
from w6a8_quantized_linear_gb300 import qlin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built()
    torch.cuda.set_device(DEV)


def chosen(score, n_keep, first=0, since=None, position=None):
    """Of one head's scores: (places that empty, tokens that move there), from the definition."""
    n = len(score)
    stays = min(n, max(0, n_keep))
    position = np.arange(n) if position is None else position
    safe = (position < first) | ((position >= since) if since is not None else False)
    key = np.where(np.isnan(score), -np.inf, score).astype(np.float64)
    order = sorted(range(n), key=lambda i: (not safe[i], -key[i], bool(np.isnan(score[i])) and not safe[i], i)
                   if not safe[i] else (False, 0.0, False, i))
    kept = np.zeros(n, bool)
    kept[order[:stays]] = True
    return stays, [i for i in range(stays) if not kept[i]], [i for i in range(stays, n) if kept[i]]


class Evict:
    def __init__(self, lens, heads, width, page, dtype=BF, layout="hnd", seed=0, room=None, positions=False, kind="spread",
                 strided=False):
        self.c = Case(lens, 1, heads, width, page, dtype, layout, seed)
        g = torch.Generator().manual_seed(seed + 1)
        B = len(lens)
        self.room = room if room is not None else max(max(lens), 0) + 3
        self.score = torch.rand(B, heads, self.room, generator=g).log_().neg_().pow_(3)
        if kind == "ties":
            self.score = (self.score * 2).floor().clamp(max=4)
        elif kind == "equal":
            self.score = torch.ones(B, heads, self.room)
        elif kind == "odd":  # every kind of number, among them both zeros and what is none
            pick = torch.tensor([0.0, -0.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 1e-45, -1e-45, 3e38, 0.1, 0.1])
            self.score = pick[torch.randint(0, len(pick), self.score.shape, generator=g)]
        elif kind == "close":  # equal but for the last bits
            self.score = torch.full_like(self.score, 1.0) + torch.randint(0, 700, self.score.shape, generator=g) * 2.0 ** -23
        self.position = None
        if positions:
            self.position = torch.stack([torch.stack([torch.randperm(self.room, generator=g) for _ in range(heads)]) for _ in range(B)]).int()
        self.strided = strided
        self.lens = lens

    def on_gpu(self, x):
        if x is None or not self.strided:
            return None if x is None else x.to(DEV)
        B, H, R = x.shape  # [heads, B, room + 5] inside
        wide = torch.zeros(H, B, R + 5, dtype=x.dtype, device=DEV)
        wide[:, :, 2:2 + R] = x.transpose(0, 1).to(DEV)
        return wide[:, :, 2:2 + R].transpose(0, 1)

    def run(self, n_keep, first=0, since=None, in_place=True, len_in_place=False, flags=0, ws=None):
        c = self.c
        B, heads = c.B, c.heads
        score, position = self.on_gpu(self.score), self.on_gpu(self.position)
        score_out = position_out = None
        if not in_place:
            score_out = torch.full((B, heads, self.room), 7.0, device=DEV)
            position_out = torch.full((B, heads, self.room), 7, dtype=torch.int32, device=DEV)
        len_out = c.step.len if len_in_place else torch.full((B,), 77, dtype=torch.int32, device=DEV)
        k0, v0 = c.k.clone(), c.v.clone()
        qlin.kv_evict(c.cache, c.step, score, i32(n_keep), first=first, since=None if since is None else i32(since),
                      position=position, score_out=score_out, position_out=position_out, len_out=len_out, ws=ws, flags=flags)
        want_k, want_v = k0.clone(), v0.clone()
        score_out = score if score_out is None else score_out
        position_out = position if position_out is None else position_out
        ws_, wp = self.score.clone(), None if self.position is None else self.position.clone()
        if not in_place:
            ws_, wp = torch.full_like(self.score, 7.0), torch.full((B, heads, self.room), 7, dtype=torch.int32)
        total = 0
        for b, n in enumerate(self.lens):
            if n < 0:
                continue
            for h in range(heads):
                pos = None if self.position is None else self.position[b, h, :n].numpy()
                stays, holes, movers = chosen(self.score[b, h, :n].numpy(), n_keep[b], first, None if since is None else since[b], pos)
                assert len(holes) == len(movers)
                total += len(holes)
                at = torch.arange(self.room, dtype=torch.int32) if pos is None else self.position[b, h]
                if not in_place:
                    ws_[b, h, :stays], wp[b, h, :stays] = self.score[b, h, :stays], at[:stays]
                if holes:
                    ws_[b, h, holes] = self.score[b, h, movers]
                    if wp is not None:
                        wp[b, h, holes] = at[movers]
                    (pf, rf), (pt, rt) = ([x[torch.tensor(i)] for x in c.places(b, 0, n)] for i in (movers, holes))
                    want_k[pt, h, rt], want_v[pt, h, rt] = k0[pf, h, rf], v0[pf, h, rf]
        same = lambda a, b: torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))  # noqa: E731
        assert same(c.k, want_k) and same(c.v, want_v)
        assert torch.equal(score_out.cpu().contiguous().view(torch.int32), ws_.view(torch.int32))
        if wp is not None:
            assert torch.equal(position_out.cpu(), wp)
        want_len = [(n if len_in_place else 77) if n < 0 else min(n, max(0, k)) for n, k in zip(self.lens, n_keep)]
        assert len_out.tolist() == want_len
        return total


CASES = [
    # lens, heads, width, page, dtype, layout, n_keep, kind, positions, first, since
    ([1], 1, 64, 16, BF, "hnd", [1], "spread", False, 0, None),
    ([1, 0], 2, 64, 16, BF, "hnd", [0, 3], "spread", False, 0, None),
    ([40, 17, -1], 3, 128, 16, FP, "nhd", [20, 16, 5], "spread", True, 0, None),
    ([4130], 8, 128, 16, BF, "hnd", [4088], "spread", True, 4, [4002]),
    ([20011], 2, 256, 64, BF, "hnd", [2500], "spread", False, 4, [19500]),
    ([9001, 7000, 300, 5], 5, 64, 32, FP, "pool", [4500, 6999, 299, 4], "ties", False, 2, [8000, 6000, 0, 5]),
    ([5000, 2049], 2, 64, 128, BF, "hnd", [1200, 2048], "odd", True, 0, None),
    ([3001], 1, 128, 256, BF, "nhd", [1500], "equal", False, 0, None),
    ([33000], 1, 64, 16, FP, "hnd", [12345], "close", False, 0, [32990]),
    ([2500], 2, 64, 32, BF, "hnd", [100], "spread", False, 60, [2400]),  # more is safe than there is room for
    ([1000, 1000], 2, 64, 32, BF, "hnd", [999, 1], "ties", True, 0, [-5, 1]),
]


@pytest.mark.parametrize("how", ["in place", "apart", "strided"])
@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_evict_against_its_definition(case, how):
    lens, heads, D, page, dtype, layout, n_keep, kind, positions, first, since = case
    e = Evict(lens, heads, D, page, dtype, layout, 5, kind=kind, positions=positions, strided=how == "strided")
    e.run(n_keep, first, since, in_place=how != "apart", len_in_place=how == "in place")


def test_evict_many_items_and_one_long_one():
    """One block per item; and a cluster whose blocks form part of their keys again."""
    Evict([200 + 7 * i for i in range(60)], 8, 64, 16, seed=9).run([100 + 5 * i for i in range(60)], 3, [190 + 7 * i for i in range(60)])
    assert Evict([700001], 1, 64, 256, FP, seed=2, kind="close").run([90001], 4, [699000], in_place=False) > 10000


def test_evict_again_and_again():
    """A cache held at its room: a token more, one fewer, by a captured call whose inputs change; the newest stay."""
    heads, room, D = 2, 64, 64
    c = Case([room], 1, heads, D, 16, BF, seed=3)
    g = torch.Generator().manual_seed(8)
    score, position = torch.rand(1, heads, room + 1, generator=g).to(DEV), torch.arange(room + 1, dtype=torch.int32, device=DEV).repeat(1, heads, 1)
    n_keep, since, length = i32([room]), i32([0]), c.step.len
    ws = qlin.new_workspace(qlin.kv_evict_workspace_bytes(c.cache, c.step, room + 1), DEV)
    call = lambda: qlin.kv_evict(c.cache, c.step, score, n_keep, since=since, position=position, len_out=length, ws=ws)  # noqa: E731
    call()  # moves nothing
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    key = [[(float(score[0, h, i]), i) for i in range(room)] for h in range(heads)]  # what each place holds: score, position
    rows = [[c.get(0, i, 1)[0][0, h] for i in range(room)] for h in range(heads)]
    for step in range(100):
        at = room + step
        new = torch.randn(1, heads, D, generator=g).bfloat16()
        c.put(0, room, new, new)
        fresh = torch.rand(heads, generator=g)
        score[0, :, room], position[0, :, room] = fresh.to(DEV), at
        since.fill_(at - 15)
        length.fill_(room + 1)
        graph.replay()
        for h in range(heads):
            key[h].append((float(fresh[h]), at))
            rows[h].append(new[0, h])
            worst = min((i for i in range(room + 1) if key[h][i][1] < at - 15), key=lambda i: (key[h][i][0], -i))
            key[h][worst], rows[h][worst] = key[h][room], rows[h][room]
            key[h].pop(), rows[h].pop()
    assert length.tolist() == [room]
    for h in range(heads):
        assert position[0, h, :room].tolist() == [k[1] for k in key[h]]
        assert torch.equal(torch.stack(rows[h]), c.get(0, 0, room)[0][:, h])


def test_evict_reports_what_it_cannot_follow():
    """Pages out of range, and more tokens than the scores or the table have room for."""
    e = Evict([100, 100, 60], 2, 64, 16, seed=1, room=90)
    c = e.c
    ws = qlin.new_workspace(qlin.kv_evict_workspace_bytes(c.cache, c.step, 90), DEV)
    k0, s0 = c.k.clone(), e.score.to(DEV)
    score, length = s0.clone(), torch.full((3,), 9, dtype=torch.int32, device=DEV)
    qlin.kv_evict(c.cache, c.step, score, i32([10, 10, 60]), len_out=length, ws=ws)
    assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX
    assert length.tolist() == [100, 100, 60] and torch.equal(score, s0)
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16))
    e = Evict([60], 1, 64, 16, seed=1)
    e.score[:] = torch.arange(63.0)  # all of the last ones stay
    c = e.c
    table = c.table.clone()
    table[0, 3] = 1 << 20
    c.step = qlin.KVStep(table.to(DEV), c.step.len, 1)
    k0 = c.k.clone()
    ws = qlin.new_workspace(qlin.kv_evict_workspace_bytes(c.cache, c.step, 63), DEV)
    qlin.kv_evict(c.cache, c.step, e.score.to(DEV), i32([30]), ws=ws)
    assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX
    for i in range(18):  # tokens 30 .. 47 have moved; those of the page out of range have not
        assert torch.equal(c.get(0, i, 1)[0], k0[c.places(0, 30 + i, 1)[0], :, c.places(0, 30 + i, 1)[1]].cpu())
    for i in range(18, 30):
        p, r = c.places(0, i, 1)
        assert torch.equal(c.get(0, i, 1)[0], k0[p, :, r].cpu())


def test_evict_on_another_stream_and_behind_another_kernel():
    e = Evict([3000, 2000], 4, 64, 16, seed=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e.run([1000, 1500], flags=qlin.FLAG_PDL)
    torch.cuda.current_stream().wait_stream(side)


def test_weights_and_eviction_past_32_bits_and_a_table_inside_a_wider_one():
    """The same tokens on the last pages of a cache of 2.3e9 elements and on a small one: the same bits."""
    heads, page, D, T, n = 4, 64, 128, 4, 300
    many = 70001  # pages of 32768 elements
    g = torch.Generator().manual_seed(3)
    k0, v0 = (torch.randn(6, heads, page, D, generator=g).to(BF).to(DEV) for _ in range(2))
    q = torch.randn(T, 8 * D, generator=g).to(BF).to(DEV)
    results = []
    for pages, order in ((6, [2, 0, 5, 1, 4, 3]), (many, [many - 1, many - 5, 66000, many - 2, 65537, 69000])):
        ck, cv = (torch.empty(pages, heads, page, D, dtype=BF, device=DEV) for _ in range(2))
        at = torch.tensor(order, device=DEV)
        ck[at], cv[at] = k0, v0
        wide = torch.full((1, 9), -3, dtype=torch.int32, device=DEV)
        wide[0, 2:8] = i32(order)
        step = qlin.KVStep(wide[:, 2:8], i32([n]), T)
        cache = qlin.KVCache(ck, cv)
        stats = torch.empty(T, 8, 2, device=DEV)
        out = qlin.tree_attention(cache, step, q, stats=stats)
        score, position = torch.zeros(1, heads, 350, device=DEV), torch.arange(350, dtype=torch.int32, device=DEV).repeat(1, heads, 1)
        qlin.kv_weigh(cache, step, q, stats, score, position_out=position)
        step.len.fill_(n + T)
        qlin.kv_evict(cache, step, score, i32([150]), since=i32([n]), position=position, len_out=step.len)
        results.append((out, stats, score, position, ck[at], cv[at], step.len.clone()))
        del ck, cv, cache, step
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_workspaces_shared_by_two_graphs_one_after_the_other():
    """Two captured evictions of other shapes on one workspace, replayed in turn."""
    parts = [Evict([900, 700], 2, 64, 16, seed=5), Evict([3000], 4, 128, 32, seed=6)]
    keep = [i32([400, 300]), i32([1000])]
    ws = qlin.new_workspace(max(qlin.kv_evict_workspace_bytes(e.c.cache, e.c.step, e.room) for e in parts), DEV)
    scores, graphs, length = [e.score.to(DEV) for e in parts], [], [torch.zeros(len(e.lens), dtype=torch.int32, device=DEV) for e in parts]
    out = [torch.zeros_like(s) for s in scores]
    for e, s, k, o, n in zip(parts, scores, keep, out, length):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qlin.kv_evict(e.c.cache, e.c.step, s, k, score_out=o, len_out=n, ws=ws)
        graphs.append(graph)
    for i in (0, 1, 1, 0):
        out[i].zero_()
        graphs[i].replay()
    for e, s, k, o, n in zip(parts, scores, keep, out, length):
        assert torch.equal(n, k)
        for b in range(len(e.lens)):
            m = int(k[b])
            want = e.score[b, :, : e.lens[b]].sort(-1, descending=True).values[:, :m]
            assert torch.equal(o[b, :, :m].cpu().sort(-1, descending=True).values, want) and (o[b, :, m:] == 0).all()


@pytest.mark.parametrize("lens, heads, room, width", [([300, 50], 2, 100000, 64), ([5000], 8, 60000, 128), ([100 + 9 * i for i in range(45)], 2, 20000, 64)],
                         ids=["0", "1", "2"])
@pytest.mark.parametrize("in_place", [False, True])
def test_room_and_table_much_wider_than_the_lengths(lens, heads, room, width, in_place):
    """As a program has them that captures its step once: clusters with hardly anything to do, keys not held in registers."""
    e = Evict(lens, heads, width, 16, seed=12, room=room, kind="ties")
    c = e.c
    table = torch.full((len(lens), -(-room // 16)), -7, dtype=torch.int32)
    table[:, : c.table.shape[1]] = c.table
    c.step = qlin.KVStep(table.to(DEV), c.step.len, 1)
    e.run([max(1, n // 3) for n in lens], 2, [n - 8 for n in lens], in_place=in_place, len_in_place=in_place)
