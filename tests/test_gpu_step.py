"""The step operators on the GPU against plain 64-bit forms (tests/step_ref.py):
append with head norms and rotation, tree attention, keep, sampling, and a run
of them together with the linears."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import DEV, built
from w6a8_quantized_linear_gb300 import inputs, qlin

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built()
    torch.cuda.set_device(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Case:
    """A cache whose every place that no token lies on holds NaN, a page table in
    random order, and a step over it."""

    def __init__(self, lens, T, heads, width, page, dtype=BF, layout="hnd", seed=0, parents=None, count=None, tree="shared",
                 fill=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.T, self.heads, self.width, self.page, self.dtype, self.count = lens, T, heads, width, page, dtype, count
        B = len(lens)
        self.B = B
        per = [max(1, -(-(max(n, 0) + T) // page)) for n in lens]
        pages = sum(per) + 2
        order = torch.randperm(pages, generator=g).tolist()
        most = max(per) + 1
        table = torch.full((B, most), -7, dtype=torch.int32)  # entries behind the last page are never read
        for b in range(B):
            table[b, : per[b]] = torch.tensor([order.pop() for _ in range(per[b])], dtype=torch.int32)
        self.table = table
        shape = (pages, heads, page, width) if layout != "nhd" else (pages, page, heads, width)
        if layout == "pool":  # k and v of several layers in one pool: slices with wide strides
            pool = torch.full((pages, 2, 3, heads, page, width), math.nan, dtype=dtype, device=DEV)
            self.k, self.v = pool[:, 0, 1], pool[:, 1, 1]
        else:
            self.k, self.v = (torch.full(shape, math.nan, dtype=dtype, device=DEV) for _ in range(2))
            if layout == "nhd":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.host = []  # each sequence's [tokens, heads, width] k and v
        for b, n in enumerate(lens):
            m = max(n, 0) + (self.used(b) if fill else 0)
            k, v = (torch.randn(m, heads, width, generator=g).to(dtype) for _ in range(2))
            self.host.append([k, v])
            if m:
                self.put(b, 0, k, v)
        parents = parents if parents is not None else [t - 1 for t in range(T)]
        depth, mask = [], []
        for t in range(T):
            depth.append(0 if parents[t] < 0 else depth[parents[t]] + 1)
            mask.append((0 if parents[t] < 0 else mask[parents[t]]) | 1 << t)
        self.depth, self.mask = depth, mask
        if tree == "none":
            td = tm = None
        else:
            td, tm = i32(depth), torch.tensor(mask, dtype=torch.int64).to(torch.int32).to(DEV)
            if tree == "each":
                td, tm = td.repeat(B, 1).contiguous(), tm.repeat(B, 1).contiguous()
        self.cache = qlin.KVCache(self.k, self.v)
        self.step = qlin.KVStep(table.to(DEV), i32(lens), T, count=None if count is None else i32(count), depth=td, mask=tm)

    def used(self, b):
        return R.rows_in_use(self.lens, self.count, self.T, b)

    def places(self, b, first, n):
        at = torch.arange(first, first + n)
        return self.table[b].long()[at // self.page].to(DEV), (at % self.page).to(DEV)

    def put(self, b, first, k, v):
        p, r = self.places(b, first, k.shape[0])
        self.k[p, :, r], self.v[p, :, r] = k.to(DEV), v.to(DEV)

    def get(self, b, first, n):
        p, r = self.places(b, first, n)
        return self.k[p, :, r].cpu(), self.v[p, :, r].cpu()

    def seen(self, b, t):
        n = max(self.lens[b], 0)
        m = torch.ones(n + self.used(b), dtype=torch.bool)
        for j in range(self.used(b)):
            m[n + j] = self.mask[t] >> j & 1
        return m


# ---- append ------------------------------------------------------------------------------------------------------

APPEND = [
    # lens, T, Hq, heads, width, page, dtype, src, rot, pairs, layout
    ([0], 1, 4, 4, 64, 16, BF, torch.float32, 64, False, "hnd"),
    ([15], 1, 24, 4, 256, 64, BF, torch.float32, 64, False, "hnd"),
    ([100, 3, 16], 8, 12, 2, 128, 16, FP, torch.float32, 128, True, "nhd"),
    ([1000003], 3, 5, 1, 128, 256, BF, torch.bfloat16, 32, False, "hnd"),
    ([7, 250], 33, 6, 3, 64, 32, FP, torch.bfloat16, 10, True, "pool"),
    ([31], 67, 8, 8, 256, 128, BF, torch.float32, 256, False, "nhd"),
    ([5], 2, 1, 1, 64, 16, BF, torch.float32, 0, False, "hnd"),
    # a head whose pairs lie in other lanes, in the lane itself, or anywhere; heads of one warp of different kinds
    ([50], 3, 3, 1, 256, 16, BF, torch.bfloat16, 128, False, "hnd"),
    ([50], 3, 7, 3, 128, 16, FP, torch.float32, 8, False, "nhd"),
    ([50, 1], 2, 9, 3, 128, 32, BF, torch.float32, 96, False, "hnd"),
    ([50], 3, 5, 1, 64, 16, BF, torch.bfloat16, 64, True, "hnd"),
    ([9, 0, 40, 17, 3], 1, 40, 5, 256, 64, FP, torch.float32, 256, True, "pool"),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"{i}" for i in range(len(APPEND))])
def test_append_against_64_bits(case):
    lens, T, Hq, heads, D, page, dtype, src, rot, pairs, layout = case
    far = max(lens) > 100000  # a far position: the page table's first entries stay unused
    c = Case([n % 1000 for n in lens] if far else lens, T, heads, D, page, dtype, layout, seed=3, fill=False, tree="none")
    parents = torch.randint(0, 5, (T,), generator=torch.Generator().manual_seed(1)).tolist()
    depth = [d + (lens[0] - c.lens[0] if far else 0) for d in parents]  # any distances do
    c.step = qlin.KVStep(c.step.page_table, c.step.len, T, depth=i32(depth))
    g = torch.Generator().manual_seed(11)
    n = len(lens) * T
    q = (torch.randn(n, Hq * D, generator=g) * 3).to(src)
    k = (torch.randn(n, heads * D, generator=g) * 0.2).to(src)
    v = torch.randn(n, heads * D, generator=g).to(src)
    qg, kg = 0.5 + torch.rand(D, generator=g), 0.5 + torch.rand(D, generator=g)
    theta = 5e5
    radians = [theta ** (-2.0 * i / rot) for i in range(rot // 2)] if rot else []
    before = [x.clone() for x in (c.k, c.v)]
    turns = qlin.rope_turns(theta, rot, device=DEV) if rot else None
    out = qlin.kv_append(c.cache, c.step, q=q.to(DEV), k=k.to(DEV), v=v.to(DEV), q_gamma=qg.to(DEV), k_gamma=kg.to(DEV),
                         eps=1e-5, turns=turns, pairs=pairs)
    assert out.dtype == dtype
    touched = torch.zeros(c.k.shape[0], c.k.shape[2], dtype=torch.bool, device=DEV)
    for b in range(c.B):
        gk, gv = c.get(b, c.lens[b], T)
        p, r = c.places(b, c.lens[b], T)
        touched[p, r] = True
        for t in range(T):
            row = b * T + t
            pos = c.lens[b] + depth[t]
            ref = R.append_row(q[row].view(Hq, D), qg, 1e-5, pos, radians, pairs)
            err = (out[row].cpu().double().view(Hq, D) - ref).abs()
            assert (err <= R.append_bound(ref, dtype)).all(), (b, t, "q", float((err - R.append_bound(ref, dtype)).max()))
            ref = R.append_row(k[row].view(heads, D), kg, 1e-5, pos, radians, pairs)
            err = (gk[t].double() - ref).abs()
            assert (err <= R.append_bound(ref, dtype)).all(), (b, t, "k", float((err - R.append_bound(ref, dtype)).max()))
            assert torch.equal(gv[t], v[row].view(heads, D).to(dtype))
    # nothing else of the cache has changed (compared as bits: it holds NaN)
    for was, now in zip(before, (c.k, c.v)):
        a, b_ = was.transpose(1, 2).contiguous().view(torch.int16), now.transpose(1, 2).contiguous().view(torch.int16)
        assert torch.equal(a[~touched], b_[~touched])


def test_append_parts_counts_and_absent_sequences():
    c = Case([4, -1, 9, 20], 3, 2, 64, 16, count=[2, 3, 0, 3], fill=False, tree="none")
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(12, h * 64, generator=g).to(DEV) for h in (4, 2, 2))
    q_out = torch.full((12, 256), 7.0, dtype=BF, device=DEV)
    before = c.k.clone()
    turns = qlin.rope_turns(1e4, 64, device=DEV)
    qlin.kv_append(c.cache, c.step, q=q, k=k, v=v, turns=turns, q_out=q_out)
    used = [0, 1, 9, 10, 11]
    rest = [r for r in range(12) if r not in used]
    assert (q_out[rest] == 7).all()
    radians = [1e4 ** (-2.0 * i / 64) for i in range(32)]
    for row in used:
        b, t = divmod(row, 3)
        ref = R.append_row(q[row].cpu().view(4, 64), None, 0, c.lens[b] + t, radians, False)
        assert ((q_out[row].cpu().double().view(4, 64) - ref).abs() <= R.append_bound(ref, BF)).all()
    written = (~c.k.isnan() & before.isnan()).any(-1).any(1).sum()  # token places
    assert written == 5
    # q alone leaves the cache, k and v alone need no q
    k0 = c.k.clone()
    only = qlin.kv_append(c.cache, c.step, q=q, turns=turns, q_out=torch.full_like(q_out, 7.0))
    assert torch.equal(only, q_out) and torch.equal(c.k.view(torch.int16), k0.view(torch.int16))
    c.k.fill_(math.nan)
    c.v.fill_(math.nan)
    assert qlin.kv_append(c.cache, c.step, k=k, v=v, turns=turns) is None
    gk, gv = c.get(3, 20, 3)
    assert not gk.isnan().any() and torch.equal(gv, v[9:].cpu().view(3, 2, 64).to(BF))


def test_append_takes_strided_rows_of_one_projection():
    # q, k and v as columns of one [rows, (Hq + 2 heads) * width] buffer
    c = Case([30], 5, 2, 128, 16, fill=False)
    x = torch.randn(5, (4 + 4) * 128, device=DEV)
    q, k, v = x[:, :512], x[:, 512:768], x[:, 768:]
    a = qlin.kv_append(c.cache, c.step, q=q, k=k, v=v)
    got = c.get(0, 30, 5)
    assert torch.equal(a, q.to(BF)) and torch.equal(got[0].flatten(1), k.cpu().to(BF)) and torch.equal(got[1].flatten(1), v.cpu().to(BF))


@pytest.mark.parametrize("rot, pairs", [(128, False), (64, False), (96, False), (128, True)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_append_in_place_of_a_bf16_projection(dtype, rot, pairs):
    """q_out is q itself, woven with k and v into one projection: what a call with memory of its own gives."""
    D, Hq, heads, T = 128, 40, 4, 70
    c = Case([50, 3], T, heads, D, 16, dtype, fill=False, tree="none")
    x = torch.randn(2 * T, (Hq + 2 * heads) * D, generator=torch.Generator().manual_seed(rot)).to(BF).to(DEV)
    q, k, v = x[:, : Hq * D], x[:, Hq * D: (Hq + heads) * D], x[:, (Hq + heads) * D:]
    kw = dict(k=k, v=v, q_gamma=torch.rand(D, device=DEV), k_gamma=torch.rand(D, device=DEV),
              turns=qlin.rope_turns(1e5, rot, device=DEV), pairs=pairs)
    want, rest = qlin.kv_append(c.cache, c.step, q=q, **kw), x[:, Hq * D:].clone()
    stored = [t.clone() for t in (c.k, c.v)]
    own = q if dtype is BF else x.view(FP)[:, : Hq * D]
    assert qlin.kv_append(c.cache, c.step, q=q, q_out=own, **kw) is own
    assert torch.equal(own, want) and torch.equal(x[:, Hq * D:], rest)
    for a, b in zip(stored, (c.k, c.v)):
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


def test_append_reports_pages_out_of_range():
    ws = qlin.new_workspace(256, DEV)
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        c = Case([20], 2, 1, 64, 16, fill=False)
        c.step.page_table[0, 1] = bad
        before = c.k.clone()
        k = torch.randn(2, 64, device=DEV)
        qlin.workspace_init(ws)
        out = qlin.kv_append(c.cache, c.step, q=k, k=k, v=k, ws=ws)
        assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX
        assert torch.equal(c.k.view(torch.int16), before.view(torch.int16)) and torch.equal(out, k.to(BF))
    c = Case([16 * 3 - 1], 1, 1, 64, 16, fill=False)  # a token behind the table
    c.step.len.fill_(16 * 50)
    qlin.workspace_init(ws)
    qlin.kv_append(c.cache, c.step, k=torch.randn(1, 64, device=DEV), v=torch.randn(1, 64, device=DEV), ws=ws)
    assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX


# ---- attention -----------------------------------------------------------------------------------------------------

TREE8 = [-1, 0, 1, 0, 3, 3, 0, 6]


def check_attention(c, Hq, q_seed=0, scale=None, q=None, **kw):
    D = c.width
    g = torch.Generator().manual_seed(q_seed)
    if q is None:
        q = torch.randn(c.B * c.T, Hq * D, generator=g).to(c.dtype)
    out = torch.full((c.B * c.T, Hq * D), 3.0, dtype=BF, device=DEV)
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, c.B, c.T, Hq), DEV)
    ws[256:] = 0xFF  # what an earlier call left must not matter: NaN everywhere
    got = qlin.tree_attention(c.cache, c.step, q.to(DEV), scale=scale, out=out, ws=ws, **kw)
    assert qlin.read_device_status(ws) == qlin.OK
    scale = D ** -0.5 if scale is None else scale
    group = Hq // c.heads
    got = got.cpu().double().view(c.B, c.T, Hq, D)
    for b in range(c.B):
        n = c.used(b)
        assert (got[b, n:] == 3).all(), "rows not in use were written"
        if n == 0:
            continue
        seen = torch.stack([c.seen(b, t) for t in range(n)])
        for h in range(c.heads):
            qq = q.view(c.B, c.T, Hq, D)[b, :n, h * group:(h + 1) * group].reshape(n * group, D)
            k, v = c.host[b][0][:, h], c.host[b][1][:, h]
            o, a, size, mass = R.attention_rows(qq, k, v, seen.repeat_interleave(group, 0), scale)
            have = got[b, :n, h * group:(h + 1) * group].reshape(n * group, D)
            far = (have - o).abs() - R.attention_bound(o, a, size, mass, D, c.dtype)
            assert not have.isnan().any() and (far <= 0).all(), (b, h, float(far.max()), float((have - o).abs().max()))
    return out


ATTENTION = [
    # lens, T, Hq, heads, width, page, dtype, layout, parents, count
    ([0], 1, 1, 1, 64, 16, BF, "hnd", None, None),
    ([1], 1, 4, 4, 128, 16, BF, "hnd", None, None),
    ([0, 5], 8, 6, 1, 256, 32, BF, "hnd", TREE8, None),
    ([15, 16, 17, 31, 32, 33], 1, 6, 2, 64, 16, FP, "nhd", None, None),
    ([63, 64, 65, 127, 128, 129], 2, 6, 2, 128, 64, BF, "hnd", None, None),
    ([255, 1, 256, 0, 257, 511], 3, 8, 1, 128, 32, FP, "pool", None, None),
    ([700, -1, 3, 0], 8, 8, 4, 64, 16, BF, "hnd", TREE8, [8, 8, 3, 0]),
    ([1333], 8, 48, 8, 128, 16, BF, "nhd", TREE8, None),
    ([1777], 1, 24, 4, 256, 64, BF, "hnd", None, None),
    ([2049], 8, 24, 4, 256, 256, FP, "hnd", TREE8, None),
    ([900], 32, 4, 1, 128, 128, BF, "hnd", [-1] + [t // 2 for t in range(31)], None),
    ([333, 90], 16, 16, 2, 64, 32, FP, "hnd", None, [16, 11]),
    ([5, 40], 1, 128, 1, 128, 16, BF, "hnd", None, None),
    ([3000, 10, 2999, 517, 1, 64, 128, 4000], 3, 16, 8, 64, 16, BF, "hnd", None, None),
    ([20011], 8, 8, 1, 128, 64, BF, "hnd", TREE8, None),
    ([9001], 1, 5, 5, 256, 16, FP, "nhd", None, None),
    # more sequences than a warp has lanes, some absent, some empty
    ([(37 * b) % 300 - (b % 7 == 3) * 1000 for b in range(45)], 2, 4, 2, 64, 16, BF, "hnd", None,
     [(b % 5 != 2) + (b % 3 != 1) for b in range(45)]),
    # 65 to 128 query rows of one cache head, every width
    ([700, 64], 9, 8, 1, 256, 16, FP, "hnd", None, None),
    ([1300], 32, 6, 2, 64, 64, BF, "nhd", [-1] + [max(0, t - 3) for t in range(31)], None),
    ([515], 11, 7, 1, 128, 32, BF, "hnd", None, None),
]


@pytest.mark.parametrize("case", ATTENTION, ids=[f"{i}" for i in range(len(ATTENTION))])
def test_attention_against_64_bits(case):
    lens, T, Hq, heads, D, page, dtype, layout, parents, count = case
    c = Case(lens, T, heads, D, page, dtype, layout, seed=7, parents=parents, count=count, tree="shared" if parents else "none")
    check_attention(c, Hq)


EVERY = [
    # lens, T, Hq, heads, width, page, dtype, parents
    ([20011], 8, 8, 1, 128, 64, BF, TREE8),
    ([130999], 8, 24, 4, 256, 64, BF, TREE8),
    ([30011, 9001, 517, 0, 22222, 1, 127, 128, 15000], 3, 48, 8, 128, 32, FP, None),
    ([9001], 1, 5, 5, 256, 16, FP, None),
    ([50001, 300], 32, 8, 2, 64, 128, BF, [-1] + [t // 2 for t in range(31)]),
    ([40003], 1, 2, 2, 64, 256, FP, None),
    ([70007, 3], 10, 10, 2, 128, 16, BF, None),
]


@pytest.mark.parametrize("case", EVERY, ids=[f"{i}" for i in range(len(EVERY))])
def test_attention_counts_every_token_once(case):
    """All keys are alike, so each of the n tokens that a row sees has the weight 1 / n, and all values are zero but for
    one token a column: that column gives 4096 / n if the row sees the token, or zero.  One call after another until every
    token of every sequence and cache head has had its column: one that is lost, doubled, or read from another place
    is off by all of its column, however long the context is."""
    lens, T, Hq, heads, D, page, dtype, parents = case
    B, group, parents = len(lens), Hq // heads, parents or [t - 1 for t in range(T)]
    g = torch.Generator().manual_seed(T)
    per = [-(-(n + T) // page) for n in lens]
    order = torch.randperm(sum(per) + 2, generator=g).to(torch.int32)
    table = torch.full((B, max(per)), -7, dtype=torch.int32)
    for b in range(B):
        table[b, : per[b]] = order[sum(per[:b]): sum(per[: b + 1])]
    table = table.to(DEV)
    k, v = (torch.full((sum(per) + 2, heads, page, D), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    tail = []  # the places behind the last token
    for b, n in enumerate(lens):
        k[table[b, : per[b]].long()] = 0.5
        tail.append((table[b, per[b] - 1].long(), n + T - (per[b] - 1) * page))
        k[tail[b][0], :, tail[b][1]:] = math.nan
    mask = [0] * T
    for t in range(T):
        mask[t] = (mask[parents[t]] if parents[t] >= 0 else 0) | 1 << t
    cache = qlin.KVCache(k, v)
    step = qlin.KVStep(table, i32(lens), T, mask=torch.tensor(mask).to(torch.int32).to(DEV))
    q = torch.randn(B * T, Hq * D, generator=g).to(dtype).to(DEV)
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(cache, B, T, Hq), DEV)
    n = torch.tensor(lens, device=DEV)[:, None, None]
    rows = torch.tensor(mask, device=DEV)
    count = torch.tensor([bin(m).count("1") for m in mask], device=DEV)
    share = (4096.0 / (n + count[None, :, None])).double()[..., None]  # [B, T, 1, 1]
    col, head = torch.arange(D, device=DEV), torch.arange(heads, device=DEV)[:, None]
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for first in range(0, max(lens) + T, heads * D):
        token = (first + head * D + col).expand(B, heads, D)
        there = token < n + T
        v.zero_()
        for page_of, at in tail:
            v[page_of, :, at:] = math.nan
        b, h, c = there.nonzero(as_tuple=True)
        at = token[b, h, c]
        v[table[b, at // page].long(), h, at % page, c] = 4096
        out = qlin.tree_attention(cache, step, q, ws=ws).view(B, T, heads, group, D).double()
        ahead = (token - n)[:, None]                                                # [B, 1, heads, D]
        bit = rows[None, :, None, None] >> ahead.clamp(0, 31) & 1 == 1
        seen = there[:, None] & ((ahead < 0) | bit)
        want = torch.where(seen, share, 0.0)[:, :, :, None]
        # half a step for the weight's rounding and for the result's, the fp32 sums and exponents
        wrong += (~((out - want).abs() <= (2 * 2.0 ** -8 + 2.0 ** -14) * want)).sum()
    assert int(wrong) == 0
    assert qlin.read_device_status(ws) == qlin.OK


def test_attention_trees_of_each_sequence_and_other_scales():
    c = Case([70, 200, 9], 8, 2, 128, 16, parents=TREE8, tree="each", seed=2)
    check_attention(c, 6, scale=0.5)
    check_attention(c, 6, scale=0.0)
    check_attention(c, 6, scale=-0.3)
    # scores far beyond the range of exp: one token takes all, or the weights underflow
    check_attention(c, 6, scale=40.0)


def test_attention_empty_rows_are_zero():
    c = Case([0, 12], 4, 2, 64, 16, parents=[-1, 0, 1, 2], seed=4)
    c.mask = [0, 2, 0, 8]
    c.step = qlin.KVStep(c.step.page_table, c.step.len, 4, mask=i32(c.mask))
    out = check_attention(c, 4)
    assert (out[0] == 0).all() and (out[2] == 0).all() and (out[1] != 0).any() and (out[4] != 0).any()


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_masked_rows_contribute_nothing(what, D):
    """A drafted row that holds NaN or infinities reaches only the rows that see it."""
    c = Case([130], 8, 2, D, 16, parents=TREE8, seed=8)
    for x in c.host[0]:
        x[130 + 4] = what  # row 4: seen by itself alone
        x[130 + 6, :, 3] = what  # row 6: seen by rows 6 and 7
    c.put(0, 0, *c.host[0])
    q = torch.randn(8, 4 * D, generator=torch.Generator().manual_seed(1)).to(BF)
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, 1, 8, 4), DEV)
    out = qlin.tree_attention(c.cache, c.step, q.to(DEV), ws=ws).cpu()
    clean = Case([130], 8, 2, D, 16, parents=TREE8, seed=8)
    want = qlin.tree_attention(clean.cache, clean.step, q.to(DEV), ws=ws).cpu()
    for t in (0, 1, 2, 3, 5):
        assert torch.equal(out[t], want[t]), t
    assert not out[4].isfinite().all()


def test_attention_adversarial_maxima():
    """Scores that rise along the cache, and jump, and a first token that dwarfs the rest."""
    c = Case([5000], 8, 1, 128, 32, parents=TREE8, seed=9)
    k, v = c.host[0]
    ramp = torch.linspace(-3, 6, k.shape[0])
    ramp[1700:1750] += 9
    k[:, 0] = (ramp[:, None] * torch.ones(128)).to(BF)
    c.put(0, 0, k, v)
    q = torch.ones(8, 8 * 128).to(BF)
    check_attention(c, 8, q=q)
    check_attention(c, 8, q=-q)
    k[0, 0] = 30
    c.put(0, 0, k, v)
    check_attention(c, 8, q=q)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("group", [1, 2, 4])
def test_attention_small_weights_add_up(group, dtype):
    """In each sequence four tokens, one in each part of the first tile, dwarf 200000 others of 2^-25.6 of their weight,
    which together weigh 0.1 % of them: as many sequences (over the same pages) as there are SMs, so that one run of
    tiles holds the whole of one.  The dwarfing tokens' values are zero, the others' one: o is the others' share."""
    n, T, D, page, w = 200000, 32, 64, 64, 2.0 ** -25.6
    B = torch.cuda.get_device_properties(DEV).multi_processor_count
    pages = n // page + 1
    k, v = torch.zeros(pages, 1, page, D, dtype=dtype, device=DEV), torch.ones(pages, 1, page, D, dtype=dtype, device=DEV)
    for token in (0, 32, 64, 96):
        k[token // page, 0, token % page] = 1
        v[token // page, 0, token % page] = 0
    table = torch.arange(pages, dtype=torch.int32, device=DEV).repeat(B, 1)
    step = qlin.KVStep(table, i32([n] * B), T, mask=i32([0] * T))
    q = torch.ones(B * T, group * D, dtype=dtype, device=DEV)
    out = qlin.tree_attention(qlin.KVCache(k, v), step, q, scale=25.6 * math.log(2) / D).double()
    others = (n - 4) * w
    want = others / (4 + others)
    # a weight is rounded by half a step (the smallest fp16 ones, 2^7 of the largest's scale, step by 2^-24: half of that
    # is 2^-32 of the largest), its exponent by 2 * 2^-24 * 25.6, the result by half a step of bf16
    each = max(R.HALF[dtype] * w, 2.0 ** -32 if dtype is FP else 0.0) + 2.0 ** -18 * w
    assert float((out - want).abs().max()) <= 2.0 ** -8 * want + (1 + 2.0 ** -8) * (n - 4) * each / 4


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("T, Hq, scale", [(1, 2, 2.0 ** 28), (4, 4, 2.0 ** 24), (16, 6, 2.0 ** 28), (20, 8, -2.0 ** 33), (3, 2, 2.0 ** 40)])
def test_attention_huge_scores_choose_the_largest(T, Hq, scale, dtype):
    """Whole-number q and k under a scale of 2^24 and more: every score but the largest (and its equals) has no weight,
    however far the fp32 scores' own steps are apart."""
    c = Case([3000, 5, 0, 700], T, 2, 128, 32, dtype, seed=T)
    g = torch.Generator().manual_seed(T)
    for b, n in enumerate(c.lens):
        k = torch.randint(-2, 3, c.host[b][0].shape, generator=g).to(dtype)
        c.host[b][0] = k
        c.put(b, 0, k, c.host[b][1])
    q = torch.randint(-2, 3, (c.B * T, Hq * 128), generator=g).to(dtype)
    got = qlin.tree_attention(c.cache, c.step, q.to(DEV), scale=scale).cpu().double().view(c.B, T, Hq, 128)
    group = Hq // 2
    for b in range(c.B):
        seen = torch.stack([c.seen(b, t) for t in range(T)]).repeat_interleave(group, 0)
        for h in range(2):
            qq = q.view(c.B, T, Hq, 128)[b, :, h * group:(h + 1) * group].reshape(T * group, 128)
            o, a, _, _ = R.attention_rows(qq, c.host[b][0][:, h], c.host[b][1][:, h], seen, scale)
            have = got[b, :, h * group:(h + 1) * group].reshape(T * group, 128)
            # the weights are one or nothing: what is rounded is their shares (2^-24 each) and the result, by half a step
            assert bool(((have - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -20 * a).all()), (b, h, float((have - o).abs().max()))


def test_attention_rows_do_not_depend_on_the_batch_values():
    c = Case([400, 77], 4, 2, 128, 16, seed=12)
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, 2, 4, 6), DEV)
    q = torch.randn(8, 6 * 128, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    a = qlin.tree_attention(c.cache, c.step, q, ws=ws)
    q2 = q.clone()
    q2[4:] = 5
    b = qlin.tree_attention(c.cache, c.step, q2, ws=ws)
    assert torch.equal(a[:4], b[:4])
    for _ in range(3):  # the same call, the same bits
        assert torch.equal(a, qlin.tree_attention(c.cache, c.step, q, ws=ws))


def test_attention_bad_pages_are_reported_and_not_followed():
    for bad in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        c = Case([200, 40], 2, 2, 64, 16, seed=3)
        c.step.page_table[0, 5] = bad
        ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, 2, 2, 4), DEV)
        q = torch.randn(4, 256, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
        out = qlin.tree_attention(c.cache, c.step, q, ws=ws)
        assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX
        good = Case([200, 40], 2, 2, 64, 16, seed=3)
        assert torch.equal(out[2:], qlin.tree_attention(good.cache, good.step, q)[2:])  # the other sequence's rows
    c = Case([40], 2, 2, 64, 16, seed=3)
    c.step.len.fill_(2 ** 31 - 5)  # a length far behind the table
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, 1, 2, 4), DEV)
    qlin.tree_attention(c.cache, c.step, torch.zeros(2, 256, dtype=BF, device=DEV), ws=ws)
    assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX


@pytest.mark.parametrize("copy", [0, 1, 2, 5, 13])
@pytest.mark.parametrize("n", [100, 150000])
def test_attention_an_expired_wait_is_reported_not_hung(n, copy):
    """A tile's keys or values that are never asked for, in a run of one tile and in one longer than the ring (a copy
    that the run does not have is not missed): the waits expire, the status word says so, and the next calls on the
    same workspace give what they gave before."""
    c = Case([n], 4, 1, 128, 64, seed=5)
    q = torch.randn(4, 8 * 128, generator=torch.Generator().manual_seed(3)).to(BF).to(DEV)
    out = torch.empty_like(q)
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, 1, 4, 8), DEV)
    want = qlin.tree_attention(c.cache, c.step, q, ws=ws)
    assert qlin.read_device_status(ws) == qlin.OK
    assert qlin.debug_tree_attention_fault(c.cache, c.step, q, out, ws, copy) == qlin.OK
    status = qlin.read_device_status(ws)
    if n == 100 and copy > 1:
        assert status == qlin.OK and torch.equal(out, want)
        return
    assert status == qlin.ERR_DEVICE_TIMEOUT
    for _ in range(2):
        assert torch.equal(qlin.tree_attention(c.cache, c.step, q, ws=ws), want)
    assert qlin.read_device_status(ws) == qlin.ERR_DEVICE_TIMEOUT  # until it is cleared
    qlin.workspace_init(ws)
    assert torch.equal(qlin.tree_attention(c.cache, c.step, q, ws=ws), want)
    assert qlin.read_device_status(ws) == qlin.OK


def test_attention_replayed_with_other_lengths():
    """One captured call serves every length that its table holds."""
    c = Case([900], 4, 2, 128, 16, seed=21)
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, 1, 4, 8), DEV)
    q = torch.randn(4, 1024, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    out = torch.empty(4, 1024, dtype=BF, device=DEV)
    qlin.tree_attention(c.cache, c.step, q, out=out, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qlin.tree_attention(c.cache, c.step, q, out=out, ws=ws)
    for n in (900, 0, 1, 128, 129, 500, 900):
        c.step.len.fill_(n)
        g.replay()
        eager = qlin.tree_attention(c.cache, c.step, q)
        assert torch.equal(out, eager), n


def test_attention_on_another_stream_and_with_strided_rows():
    c = Case([300], 4, 2, 64, 32, seed=5)
    buf = torch.randn(4, 3 * 256, generator=torch.Generator().manual_seed(3)).to(BF).to(DEV)
    want = qlin.tree_attention(c.cache, c.step, buf[:, 256:512].contiguous())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    wide = torch.zeros(4, 768, dtype=BF, device=DEV)
    torch.cuda.synchronize()
    got = qlin.tree_attention(c.cache, c.step, buf[:, 256:512], out=wide[:, 256:512], stream=s)
    alloc = qlin.tree_attention(c.cache, c.step, buf[:, 256:512], stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(alloc, want)
    assert (wide[:, :256] == 0).all() and (wide[:, 512:] == 0).all()


def test_attention_workspace_shared_by_two_graphs_and_two_streams_apart():
    """Two captured calls of different shapes on one workspace, replayed in turn;
    and two calls at once, each with its own."""
    a, b = Case([700], 4, 2, 128, 16, seed=1), Case([90, 1500, 33], 2, 1, 256, 64, seed=2)
    qa = torch.randn(4, 8 * 128, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    qb = torch.randn(6, 5 * 256, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    want = [qlin.tree_attention(c.cache, c.step, q).clone() for c, q in ((a, qa), (b, qb))]
    need = max(qlin.tree_attention_workspace_bytes(a.cache, 1, 4, 8), qlin.tree_attention_workspace_bytes(b.cache, 3, 2, 5))
    ws = qlin.new_workspace(need, DEV)
    outs, graphs = [torch.empty_like(w) for w in want], []
    for (c, q), o in zip(((a, qa), (b, qb)), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qlin.tree_attention(c.cache, c.step, q, out=o, ws=ws, flags=qlin.FLAG_PDL)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in (graphs[0], graphs[1], graphs[1], graphs[0]):
            g.replay()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [qlin.new_workspace(need, DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for (c, q), o, s, w in zip(((a, qa), (b, qb)), outs, streams, wss):
            qlin.tree_attention(c.cache, c.step, q, out=o, ws=w, stream=s, flags=qlin.FLAG_PDL)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_attention_layer_after_layer_on_one_workspace():
    """Calls in a row under programmatic dependent launch, each reading the last one's output."""
    c = Case([600], 8, 4, 128, 16, seed=15, parents=TREE8)
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, 1, 8, 8), DEV)
    q0 = torch.randn(8, 1024, generator=torch.Generator().manual_seed(4)).to(BF).to(DEV)

    def run(flags):
        x = q0
        for _ in range(12):
            x = qlin.tree_attention(c.cache, c.step, x, ws=ws, flags=flags)
        return x

    want = run(0)
    for _ in range(3):
        assert torch.equal(run(qlin.FLAG_PDL), want)


def test_the_first_call_of_a_process_may_be_captured():
    code = """
import torch
from w6a8_quantized_linear_gb300 import qlin
dev = torch.device("cuda:0")
k = torch.randn(8, 2, 16, 64, device=dev).bfloat16()
cache = qlin.KVCache(k, k.clone())
step = qlin.KVStep(torch.arange(8, dtype=torch.int32, device=dev)[None], torch.tensor([70], dtype=torch.int32, device=dev), 2)
q = torch.randn(2, 256, device=dev)
kv = torch.randn(2, 128, device=dev)
logits, u = torch.randn(3, 40000, device=dev), torch.rand(3, device=dev)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    h = qlin.kv_append(cache, step, q=q, k=kv, v=kv)
    out = qlin.tree_attention(cache, step, h)
    token = qlin.sample(logits, u)
g.replay()
torch.cuda.synchronize()
assert torch.equal(out, qlin.tree_attention(cache, step, qlin.kv_append(cache, step, q=q, k=kv, v=kv)))
assert torch.equal(token, qlin.sample(logits, u))
print("captured first")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=280)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


# ---- keep ------------------------------------------------------------------------------------------------------------

KEEP = [([10], 8, 2, 128, 16, BF, "hnd", [[0, 3, 5, 7]]), ([0, 31, 500, -1, 7], 32, 5, 64, 32, FP, "nhd",
        [[1, 2, 30, 31], list(range(32)), [], [0, 1], [31]]), ([1, 14], 5, 8, 256, 16, BF, "pool", [[0, 4], [2, 3, 4]])]


@pytest.mark.parametrize("case", KEEP, ids=["0", "1", "2"])
def test_keep_moves_the_accepted_rows(case):
    lens, T, heads, D, page, dtype, layout, kept = case
    c = Case(lens, T, heads, D, page, dtype, layout, seed=6)
    keep = torch.full((len(lens), T), 99, dtype=torch.int32)
    for b, rows in enumerate(kept):
        keep[b, : len(rows)] = torch.tensor(rows, dtype=torch.int32)
    ws = qlin.new_workspace(256, DEV)
    out = torch.full((len(lens),), -5, dtype=torch.int32, device=DEV)
    qlin.kv_keep(c.cache, c.step, keep.to(DEV), i32([len(r) for r in kept]), len_out=out, ws=ws)
    assert qlin.read_device_status(ws) == qlin.OK
    for b, rows in enumerate(kept):
        if lens[b] < 0:
            assert out[b] == -5
            continue
        assert out[b] == lens[b] + len(rows)
        for i, x in enumerate(c.get(b, 0, lens[b] + T)):
            want = c.host[b][i].clone()
            want[lens[b]: lens[b] + len(rows)] = c.host[b][i][[lens[b] + r for r in rows]]
            assert torch.equal(x, want)


def test_keep_in_place_lengths_and_bad_lists():
    ws = qlin.new_workspace(256, DEV)
    lists = [[0, 2], [2, 1], [0, 0], [1, 4], [-1, 2], [0, 1], [3, 3]]
    counts = [2, 2, 2, 2, 2, 5, -1]
    c = Case([20] * len(lists), 4, 2, 64, 16, seed=6)
    keep = torch.zeros(len(lists), 4, dtype=torch.int32)
    keep[:, :2] = torch.tensor(lists, dtype=torch.int32)
    qlin.kv_keep(c.cache, c.step, keep.to(DEV), i32(counts), len_out=c.step.len, ws=ws)
    assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX
    assert c.step.len.tolist() == [22] + [20] * (len(lists) - 1)
    for b in range(1, len(lists)):
        for x, y in zip(c.get(b, 0, 24), c.host[b]):
            assert torch.equal(x, y)
    qlin.kv_keep(c.cache, c.step, keep.to(DEV), i32([1] + [0] * (len(lists) - 1)), len_out=c.step.len)
    assert c.step.len.tolist() == [23] + [20] * (len(lists) - 1)


def test_offsets_past_32_bits_and_a_table_inside_a_wider_one():
    """The same step on the last pages of a cache of 2.3e9 elements and on a small
    one, through a table that is a slice of a wider one: the same bits."""
    heads, page, D, T, n = 4, 64, 128, 4, 300
    many = 70001  # pages of 32768 elements
    g = torch.Generator().manual_seed(3)
    k0, v0 = (torch.randn(6, heads, page, D, generator=g).to(BF).to(DEV) for _ in range(2))
    q, k, v = (torch.randn(T, h * D, generator=g).to(DEV) for h in (8, heads, heads))
    turns = qlin.rope_turns(1e6, D, device=DEV)
    results = []
    for pages, order in ((6, [2, 0, 5, 1, 4, 3]), (many, [many - 1, many - 5, 66000, many - 2, 65537, 69000])):
        ck, cv = (torch.empty(pages, heads, page, D, dtype=BF, device=DEV) for _ in range(2))
        ck[torch.tensor(order, device=DEV)], cv[torch.tensor(order, device=DEV)] = k0, v0
        wide = torch.full((1, 9), -3, dtype=torch.int32, device=DEV)
        wide[0, 2:8] = i32(order)
        step = qlin.KVStep(wide[:, 2:8], i32([n]), T, depth=i32([0, 1, 1, 2]), mask=i32([1, 3, 5, 13]))
        cache = qlin.KVCache(ck, cv)
        h = qlin.kv_append(cache, step, q=q, k=k, v=v, turns=turns)
        out = qlin.tree_attention(cache, step, h)
        qlin.kv_keep(cache, step, i32([[0, 2, 3, 0]]), i32([3]), len_out=step.len)
        at = torch.tensor(order, device=DEV)
        results.append((h, out, ck[at], cv[at], step.len.clone()))
        del ck, cv, cache, step
    for a, b in zip(*results):
        assert torch.equal(a, b)


# ---- sample ----------------------------------------------------------------------------------------------------------

def logits_of(M, V, seed, dtype=torch.float32, banned=0.0, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, V, generator=g) * spread
    x.scatter_(1, torch.randint(0, V, (M, 8), generator=g), 6 + 5 * torch.rand(M, 8, generator=g))
    if banned:
        x.masked_fill_(torch.rand(M, V, generator=g) < banned, -math.inf)
    return x.to(dtype), torch.rand(M, generator=g)


def check_sample(x, u, **kw):
    M = x.shape[0]
    dev = {n: None if t is None else t.to(DEV) for n, t in kw.items()}
    prob = torch.full((M,), -1.0, device=DEV)
    token = qlin.sample(x.to(DEV), u.to(DEV), prob=prob, **dev)
    rows = x.double().numpy()
    for m in range(M):
        pick = {n: float(t[m]) if n != "top_k" else int(t[m]) for n, t in kw.items() if t is not None}
        want, p = R.sample_row(rows[m], float(u[m]), **pick)
        assert int(token[m]) == want, (m, pick, float(u[m]), int(token[m]), want)
        # weights within 2^-31 of theirs or half of 2^-42, sums of them, rounded to fp32
        assert abs(float(prob[m]) - p) <= 2.0 ** -24 * p + 2.0 ** -29 * p + 2.0 ** -42 * len(rows[m]), (m, float(prob[m]), p)
    return token


SIZES = [1, 2, 31, 33, 1000, 4096, 4097, 32000, 50001, 131071, 262144, 300007, 524288]


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_sample_against_64_bits(V, dtype):
    M = 4
    x, u = logits_of(M, V, V, dtype)
    f = torch.tensor
    check_sample(x, u)
    check_sample(x, u, temperature=f([0.7, 1.3, 0.0, 5.0]))
    check_sample(x, u, top_k=f([1, 50, 0, V + 3], dtype=torch.int32))
    check_sample(x, u, top_p=f([0.9, 0.5, 1.0, 0.999]), temperature=f([1.0, 2.0, 0.9, 30.0]))
    check_sample(x, u, min_p=f([0.05, 0.3, 0.0, 1.0]))
    check_sample(x, u, temperature=f([0.8, 1.0, 1.2, 3.0]), top_k=f([40, 400, 7, 3], dtype=torch.int32),
                 top_p=f([0.95, 0.8, 0.3, 0.99]), min_p=f([0.02, 0.01, 0.1, 0.0]))


@pytest.mark.parametrize("V", [30000, 140001])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_sample_many_kept_tokens(V, dtype):
    """Counts on both sides of what one CTA carries on alone, and masses that reach far down."""
    x, u = logits_of(6, V, V + 1, dtype, banned=0.2, spread=0.3)
    f = torch.tensor
    k = f([1023, 1024, 1025, 2049, V // 3, V // 2], dtype=torch.int32)
    check_sample(x, u, top_k=k)
    check_sample(x, u, top_k=k, top_p=f([0.99, 0.999, 0.5, 0.9, 0.97, 0.2]), temperature=f([9.0, 1.0, 20.0, 3.0, 50.0, 7.0]))
    check_sample(x, u, top_p=f([0.9999, 0.999999, 0.99, 1 - 2.0 ** -24, 0.7, 0.01]), temperature=f([9.0, 1.0, 20.0, 3.0, 50.0, 7.0]))


def test_sample_a_large_batch_of_small_rows():
    x, u = logits_of(3001, 257, 77)
    check_sample(x, u, top_p=torch.full((3001,), 0.8))


def test_sample_many_rows_and_banned_tokens():
    x, u = logits_of(70, 5003, 1, banned=0.4)
    g = torch.Generator().manual_seed(9)
    check_sample(x, u, temperature=torch.rand(70, generator=g) * 2, top_k=torch.randint(-3, 6000, (70,), generator=g, dtype=torch.int32),
                 top_p=torch.rand(70, generator=g) * 1.2, min_p=torch.rand(70, generator=g) * 0.2 - 0.05)


@pytest.mark.parametrize("V", [5, 1000, 40000])
def test_sample_ties_go_to_the_lowest_index(V):
    """Few distinct values: every border runs through equal logits."""
    g = torch.Generator().manual_seed(V)
    x = torch.randint(0, 3, (8, V), generator=g).float() * 0.5
    x[7] = 1.25  # all equal
    u = torch.rand(8, generator=g)
    k = torch.tensor([1, 2, V // 2 + 1, V - 1, 3, V // 3 + 1, 2, V // 2], dtype=torch.int32)
    check_sample(x, u, top_k=k)
    check_sample(x, u, top_p=torch.tensor([0.1, 0.37, 0.5, 0.9, 0.99, 0.71, 0.013, 0.33]))
    check_sample(x, u, top_k=k, top_p=torch.tensor([0.1, 0.37, 0.5, 0.9, 0.99, 0.71, 0.013, 0.33]))
    check_sample(x, u, min_p=torch.tensor([1.0, 0.99, 0.5, 0.36, 0.2, 0.7, 2.0, 1.0]))
    check_sample(x, u, temperature=torch.zeros(8))


@pytest.mark.parametrize("V", [4097, 40000, 131071])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_sample_uneven_rows(V, dtype):
    """The likely tokens all in one place, or few allowed ones: what the row's parts hand on is far from even."""
    x, u = logits_of(8, V, V + 3)
    x[0] = x[0].sort(descending=True).values
    x[1] = x[1].sort().values
    x[2, torch.arange(V) % (V // 5) != 7] = -math.inf  # five or six are allowed
    x[3, V // 2: V // 2 + 300] += 20
    x[4, : V // 2] = -math.inf
    x[5] = -9.0
    x[5, V - 3:] = 4.0
    x[6, V // 3: V // 3 + 70] = math.inf
    x[7, 128:] -= 40
    x = x.to(dtype)
    f = torch.tensor
    for k in ([1, 1, 3, 1, 1, 2, 1, 1], [100, 90, 400, 250, 33, 5, 69, 127], [900, 1024, 2, 301, 1000, 700, 71, 128]):
        k = f(k, dtype=torch.int32)
        check_sample(x, u, top_k=k)
        check_sample(x, u, top_k=k, top_p=f([0.9, 0.99, 0.8, 0.999, 0.5, 0.95, 0.7, 0.97]), temperature=f([1.0, 0.7, 9.0, 2.0, 1.0, 3.0, 1.0, 20.0]),
                     min_p=f([0.0, 0.1, 0.0, 0.02, 0.3, 0.0, 0.0, 0.0]))


@pytest.mark.parametrize("n", [100, 128, 129, 600])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_sample_ties_among_the_likely(n, dtype):
    """Borders of both filters inside a run of equal likely tokens, short and long."""
    V = 40000
    x, u = logits_of(6, V, n, dtype)
    g = torch.Generator().manual_seed(n)
    for m in range(6):
        x[m, torch.randperm(V, generator=g)[:n]] = 9.25
        x[m, torch.randperm(V, generator=g)[:3]] = 10.5
    f = torch.tensor
    k = f([n // 2, n - 1, n + 3, n + 60, 2, 900], dtype=torch.int32)
    for t in ([1.0] * 6, [0.8, 1.0, 3.0, 1.3, 0.5, 1.0]):
        check_sample(x, u, temperature=f(t), top_k=k)
        check_sample(x, u, temperature=f(t), top_k=k, top_p=f([0.5, 0.9, 0.999, 0.4, 0.9, 0.7]), min_p=f([0.0, 0.1, 0.0, 0.4, 0.0, 0.2]))
        check_sample(x, u, temperature=f(t), top_p=f([0.01, 0.05, 0.1, 0.3, 0.02, 0.5]))


@pytest.mark.parametrize("V, n", [(300, 129), (2000, 700), (2048, 2048), (8001, 3000)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_sample_borders_inside_long_runs_of_one_logit(V, n, dtype):
    """Rows that one CTA takes (8001 tokens too, in so many rows), the border of either filter inside a bin of more than
    128 equal logits: the bin's range of keys and the places of its equal tokens are found one after the other.  Every
    row's answer, and the same in each of many launches."""
    M = 200
    g = torch.Generator().manual_seed(V + n)
    x = torch.randn(M, V, generator=g)
    run = torch.rand(M, V, generator=g).argsort(1)[:, :n]
    x.scatter_(1, run, 4.25)  # above nearly all others
    x = x.to(dtype)
    u = torch.rand(M, generator=g)
    k = torch.randint(max(1, n // 8), n, (M,), generator=g, dtype=torch.int32)
    p = 0.02 + 0.5 * torch.rand(M, generator=g)
    for kw in (dict(top_k=k), dict(top_p=p), dict(top_k=k, top_p=p)):
        want = check_sample(x, u, **kw)
        dev = {name: t.to(DEV) for name, t in kw.items()}
        dx, du = x.to(DEV), u.to(DEV)
        again = [qlin.sample(dx, du, **dev) for _ in range(20)]
        assert all(torch.equal(want, t) for t in again)


@pytest.mark.parametrize("M, V, dtype", [(44, 100003, torch.float32), (20, 140001, torch.float32), (20, 300007, BF), (66, 90001, torch.float32),
                                         (16, 262143, torch.float32)])
def test_sample_many_long_rows(M, V, dtype):
    """More than the SMs hold at a time, rows at every alignment, each kind of row among them."""
    x, u = logits_of(M, V, V + 5, dtype)
    inf = math.inf
    x[0, V // 2] = math.nan
    x[1] = -inf
    x[2, ::30011] = inf
    x[3] = x[3].sort(descending=True).values
    x[4] = x[4].sort().values
    x[5, torch.arange(V) % (V // 5) != 7] = -inf
    x[6] = 0.75
    x[7] = (x[7] * 0.5).round()
    x[8, ::2] = -0.0
    x[9] *= 1e-30
    x[10, V - 1] = 60.0
    g = torch.Generator().manual_seed(V)
    t = 0.5 + torch.rand(M, generator=g)
    t[11] = 0
    k = torch.randint(1, 1500, (M,), generator=g, dtype=torch.int32)
    k[12], k[13], k[14] = 0, V // 3, 1
    p = 0.3 + 0.7 * torch.rand(M, generator=g)
    q = 0.2 * torch.rand(M, generator=g)
    check_sample(x, u, temperature=t)
    check_sample(x, u, top_k=k)
    check_sample(x, u, temperature=t, top_p=p)
    check_sample(x, u, temperature=t, top_k=k, top_p=p, min_p=q)


def test_sample_edges():
    inf, nan = math.inf, math.nan
    rows = [[-inf] * 5, [0, 1, nan, 2, 3], [inf, 0, inf, 1, -inf], [-inf, -inf, 4, -inf, -inf], [3e38, -3e38, 0, 3e38, 1e38],
            [-0.0, 0.0, -0.0, 0.0, -1.0], [1e-40, 2e-40, 0, -1e-40, 1e-45], [-1e30, -1e30, -2e30, -3e30, -inf],
            [88.0, -88.0, 87.5, 0.0, 1.0], [inf, nan, 0, 0, 0]]
    x = torch.tensor(rows)
    M = len(rows)
    one = lambda v: torch.full((M,), float(v))  # noqa: E731
    for u in (0.0, 0.3, 0.5, 0.75, 1 - 2.0 ** -24, 1.0, -2.0, 7.0):
        for kw in ({}, dict(top_k=torch.full((M,), 2, dtype=torch.int32)), dict(top_p=one(0.6)), dict(top_p=one(0.0)), dict(top_p=one(-1)),
                   dict(top_p=one(nan)), dict(min_p=one(0.9)), dict(min_p=one(nan)), dict(temperature=one(0)), dict(temperature=one(-1)),
                   dict(temperature=one(nan)), dict(temperature=one(1e-30)), dict(temperature=one(1e30)),
                   dict(top_k=torch.full((M,), 3, dtype=torch.int32), top_p=one(0.9), min_p=one(0.1))):
            check_sample(x, one(u), **kw)
    t = qlin.sample(x.to(DEV), one(0.5).to(DEV), temperature=one(inf).to(DEV))  # every token that is not forbidden, alike
    assert t.tolist()[:4] == [-1, -1, 2, 2] and int(t[8]) == 2


@pytest.mark.parametrize("V", [5, 3001, 40000])
def test_sample_differences_beyond_fp32(V):
    """Rows whose logits are finite and their differences are not, at temperatures that leave them weights; infinite ones."""
    g = torch.Generator().manual_seed(V)
    M = 6
    x = (torch.rand(M, V, generator=g) * 2 - 1) * 3e38
    x[:, :2] = torch.tensor([3e38, -3e38])
    x[3, 2::3] = -math.inf
    u = torch.rand(M, generator=g)
    one = lambda v: torch.full((M,), float(v))  # noqa: E731
    k = torch.full((M,), V // 2 + 1, dtype=torch.int32)
    prob = torch.empty(M, device=DEV)
    for T in (1e38, 6e37):
        for kw in ({}, dict(top_p=one(0.9)), dict(top_k=k, min_p=one(0.01))):
            kw["temperature"] = one(T)
            token = qlin.sample(x.to(DEV), u.to(DEV), prob=prob, **{n: t.to(DEV) for n, t in kw.items()})
            for m in range(M):
                want, p = R.sample_row(x[m].double().numpy(), float(u[m]), **{n: t[m].item() for n, t in kw.items()})
                # 1 / T is a multiple of 2^-149 above 2^-127: off by 2^-24 of itself in either of two terms, and an exponent
                # of up to 6e38 / T = 10 by ten times that
                assert int(token[m]) == want and abs(float(prob[m]) - p) <= 2.0 ** -19 * p, (T, m, int(token[m]), want)
    token = qlin.sample(x.to(DEV), u.to(DEV), temperature=one(math.inf).to(DEV), prob=prob).cpu()
    for m in range(M):  # all that are not forbidden, alike
        alive = x[m].isfinite().nonzero().flatten()
        want = int(alive[min(int(float(u[m]) * len(alive)), len(alive) - 1)])
        assert int(token[m]) == want and float(prob[m]) == pytest.approx(1 / len(alive), rel=2.0 ** -22), m


def test_sample_strided_rows_and_replay():
    x, u = logits_of(3, 9001, 4)
    wide = torch.full((3, 20000), math.nan)
    wide[:, 7:9008] = x
    wide = wide.to(DEV)
    top_p = torch.tensor([0.9, 0.8, 0.7]).to(DEV)
    want = check_sample(x, u, top_p=top_p.cpu())
    assert torch.equal(want, qlin.sample(wide[:, 7:9008], u.to(DEV), top_p=top_p))
    du, token = u.to(DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qlin.sample(wide[:, 7:9008], du, top_p=top_p, token=token)
    for i in range(5):
        fresh = torch.rand(3, generator=torch.Generator().manual_seed(i))
        du.copy_(fresh)
        g.replay()
        assert torch.equal(token, check_sample(x, fresh, top_p=top_p.cpu()))


def test_sample_frequencies_follow_the_weights():
    """A grid of uniform numbers: each token's share of them is its probability."""
    n = 4096
    x = torch.tensor([[0.0, 1.0, -1.0, 2.0, -math.inf, 0.5]]).repeat(n, 1)
    u = (torch.arange(n) + 0.5) / n
    got = torch.bincount(qlin.sample(x.to(DEV), u.to(DEV)).cpu().long(), minlength=6).double() / n
    assert (got - torch.softmax(x[0].double(), 0)).abs().max() <= 1.0 / n + 1e-9  # a share's ends fall between grid points


# ---- together --------------------------------------------------------------------------------------------------------

def test_a_verification_step_with_the_linears():
    """qkv linear -> append -> tree attention -> o linear -> logits linear -> sample
    -> keep, eager and as one replayed graph, against 64-bit forms of each part on
    the bits the part before it gave; and the kept cache equals one into which
    only the accepted rows were appended."""
    K, D, Hq, heads, V, T, page = 512, 128, 8, 2, 1040, 8, 16
    n0 = 45
    kept_rows = [0, 3, 5]
    ws = qlin.new_workspace(256, DEV)

    def weight(N, Kw, seed):
        cs = inputs.make_case("w4a8", "none", 1, N, Kw, 128, seed=seed)
        w = cs.wbuf.to(DEV)
        qlin.repack(w, "w4a8", N, Kw, 128)
        return w

    Ns = [Hq * D, heads * D, heads * D]
    wqkv = [weight(N, K, 10 + i) for i, N in enumerate(Ns)]
    wo, wv = weight(K, Hq * D, 20), weight(V, K, 21)
    gamma = torch.rand(K, device=DEV) + 0.5
    qg, kg = (torch.rand(D, device=DEV) + 0.5 for _ in range(2))
    turns = qlin.rope_turns(1e6, D, device=DEV)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, K, generator=g).to(BF).to(DEV)
    u = torch.rand(T, generator=g).to(DEV)
    top_p = torch.full((T,), 0.9, device=DEV)
    c = Case([n0], T, heads, D, page, seed=30, parents=TREE8, fill=False)
    start = [t.clone() for t in (c.k, c.v)]
    aws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, 1, T, Hq), DEV)
    keep = torch.zeros(1, T, dtype=torch.int32)
    keep[0, :3] = torch.tensor(kept_rows, dtype=torch.int32)
    keep, n_keep = keep.to(DEV), i32([3])
    y = [torch.empty(T, N, device=DEV) for N in Ns]
    q, att = torch.empty(T, Hq * D, dtype=BF, device=DEV), torch.empty(T, Hq * D, dtype=BF, device=DEV)
    h, logits = torch.empty(T, K, device=DEV), torch.empty(T, V, device=DEV)
    token = torch.empty(T, dtype=torch.int32, device=DEV)

    def run(flags):
        qlin.forward_multi("w4a8", "rmsnorm", wqkv, Ns, K, 128, x=x, gamma=gamma, y=y, ws=ws, flags=flags)
        qlin.kv_append(c.cache, c.step, q=y[0], k=y[1], v=y[2], q_gamma=qg, k_gamma=kg, turns=turns, q_out=q, ws=ws, flags=flags)
        qlin.tree_attention(c.cache, c.step, q, out=att, ws=aws, flags=flags)
        qlin.forward("w4a8", "none", wo, K, Hq * D, 128, x=att, y=h, ws=ws, flags=flags)
        h16 = (h * 0.01).to(BF)
        qlin.forward("w4a8", "rmsnorm", wv, V, K, 128, x=h16, gamma=gamma, y=logits, ws=ws)
        qlin.sample(logits, u, top_p=top_p, token=token, flags=flags)
        qlin.kv_keep(c.cache, c.step, keep, n_keep, len_out=c.step.len, ws=ws, flags=flags)

    run(0)
    results = [t.clone() for t in (*y, q, att, h, logits, token)]
    assert qlin.read_device_status(ws) == qlin.OK and qlin.read_device_status(aws) == qlin.OK
    assert int(c.step.len[0]) == n0 + 3
    # the parts against 64 bits
    radians = [1e6 ** (-2.0 * i / D) for i in range(D // 2)]
    ks = []
    for t in range(T):
        pos = n0 + c.depth[t]
        ref = R.append_row(y[0][t].cpu().view(Hq, D), qg.cpu(), 1e-6, pos, radians, False)
        assert ((q[t].cpu().double().view(Hq, D) - ref).abs() <= R.append_bound(ref, BF)).all()
        ks.append(R.append_row(y[1][t].cpu().view(heads, D), kg.cpu(), 1e-6, pos, radians, False))
    got_k, got_v = c.get(0, n0, 3)
    for i, r in enumerate(kept_rows):
        assert ((got_k[i].double() - ks[r]).abs() <= R.append_bound(ks[r], BF)).all()
        assert torch.equal(got_v[i], y[2][r].cpu().view(heads, D).to(BF))
    for m in range(T):
        want, _ = R.sample_row(logits[m].double().cpu().numpy(), float(u[m]), top_p=float(top_p[m]))
        assert int(token[m]) == want
    # the accepted rows alone, appended as a chain of three, give the same cache and attention bits
    after = [t.clone() for t in (c.k, c.v)]
    chain = Case([n0], 3, heads, D, page, seed=30, fill=False, tree="none")
    chain.table[0] = c.table[0][: chain.table.shape[1]]
    chain.k, chain.v = start[0].clone(), start[1].clone()
    chain.cache = qlin.KVCache(chain.k, chain.v)
    chain.step = qlin.KVStep(c.step.page_table, i32([n0]), 3)
    sel = torch.tensor(kept_rows, device=DEV)
    q3 = qlin.kv_append(chain.cache, chain.step, q=y[0][sel].contiguous(), k=y[1][sel].contiguous(), v=y[2][sel].contiguous(),
                        q_gamma=qg, k_gamma=kg, turns=turns)
    # row 3 stands at depth 1, row 5 at depth 2: the same positions as the chain's
    assert [c.depth[r] for r in kept_rows] == [0, 1, 2] and torch.equal(q3, q[sel])
    for a, b in zip(c.get(0, 0, n0 + 3), chain.get(0, 0, n0 + 3)):
        assert torch.equal(a, b)
    # one graph of the whole step, with and without programmatic dependent launch
    for flags in (0, qlin.FLAG_PDL):
        c.step.len.fill_(n0)
        c.k.copy_(start[0]), c.v.copy_(start[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(flags)
        for t in (*y, q, att, h, logits):
            t.zero_()
        graph.replay()
        for a, b in zip(results, (*y, q, att, h, logits, token)):
            assert torch.equal(a, b)
        assert int(c.step.len[0]) == n0 + 3
        for a, b in zip(after, (c.k, c.v)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
