"""Accumulated attention weights on the GPU against a plain 64-bit form, and the softmax statistics that they come from."""
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


def rows_of(c, q, b, h, Hq):
    """Sequence b's query rows of cache head h: [T, group, D] in 64 bits."""
    return q.view(c.B, c.T, c.heads, Hq // c.heads, c.width)[b, :, h].cpu().double()


def attend(c, q, Hq, scale=None):
    """tree_attention with its statistics."""
    stats = torch.full((c.B * c.T, Hq, 2), 7.0, device=DEV)
    out = qlin.tree_attention(c.cache, c.step, q, stats=stats, scale=scale)
    return out, stats


def reference(c, q, stats, Hq, b, h, path=None, scale=None):
    """Weights of the committed tokens and of the kept rows' own, in 64 bits, and the bound on their errors: per weight, the
    score's (D + 8) 2^-24 sum |q| |k| scale (log2 units 1.45 of it, twice for the weight's relative error: 3), its reference's
    and the exponent's rounding (2^-23 of the exponent's size, then ex2: 2^-21), the products (4 2^-24), and fp32 sums of
    `group` weights per row (2^-24 each, of the sum)."""
    n, D = max(c.lens[b], 0), c.width
    scale = D ** -0.5 if scale is None else scale
    k = c.host[b][0][:, h].double()
    keep = list(range(c.used(b))) if path is None else path
    tokens = list(range(n)) + [n + r for r in keep]
    qq, st = rows_of(c, q, b, h, Hq), stats.view(c.B, c.T, c.heads, Hq // c.heads, 2)[b, :, h].cpu().double()
    total, err = torch.zeros(len(tokens), dtype=torch.float64), torch.zeros(len(tokens), dtype=torch.float64)
    count = 0
    for i, t in enumerate(keep):
        seen = torch.ones(len(tokens), dtype=torch.bool)
        for j, r in enumerate(keep):
            seen[n + j] = (j <= i) if path is not None else bool(c.mask[t] >> r & 1)
        kk = torch.where(seen[:, None], k[tokens], 0)
        x = (qq[t] @ kk.T) * scale * math.log2(math.e)
        size = (qq[t].abs() @ kk.abs().T) * abs(scale)
        w = torch.where(seen, torch.exp2(x - st[t, :, :1]) / st[t, :, 1:], 0)
        rel = 3 * (D + 8) * 2.0 ** -24 * size + 2.0 ** -23 * (x.abs() + st[t, :, :1].abs()) + 2.0 ** -21 + 4 * 2.0 ** -24
        total += w.sum(0)
        err += (w * rel).sum(0)
        count += w.shape[0]
    return total, err + (count + 4) * 2.0 ** -24 * total + 1e-37


CASES = [
    # lens, T, Hq, heads, width, page, dtype, layout, count, path, parents
    ([1], 1, 1, 1, 64, 16, BF, "hnd", None, None, None),
    ([0], 1, 4, 4, 128, 16, FP, "hnd", None, None, None),
    ([1777], 1, 24, 4, 256, 64, BF, "hnd", None, None, None),
    ([300, 0, 127, 128, 129], 5, 6, 2, 128, 32, FP, "nhd", [5, 3, 0, 1, 5], None, [-1, 0, 0, 1, 3]),
    ([1000, 40, -1, 517], 8, 8, 2, 64, 16, BF, "pool", None, [[0, 2, 5], [0], [0], []], [-1, 0, 0, 1, 2, 2, 4, 4]),
    ([640, 2000], 16, 16, 2, 128, 128, BF, "hnd", None, None, None),
    ([4001], 32, 4, 1, 256, 256, FP, "hnd", None, [list(range(0, 32, 3))], [-1] + list(range(31))),
    ([333] * 9, 3, 15, 5, 64, 16, BF, "hnd", None, [[0, 1, 2]] * 9, [-1, 0, 1]),
    ([20000, 11], 2, 12, 3, 128, 64, BF, "nhd", None, None, [-1, -1]),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
@pytest.mark.parametrize("apart", [False, True], ids=["in place", "apart"])
def test_weigh_against_64_bits(case, apart):
    lens, T, Hq, heads, D, page, dtype, layout, count, paths, parents = case
    c = Case(lens, T, heads, D, page, dtype, layout, seed=6, count=count, parents=parents)
    g = torch.Generator().manual_seed(7)
    q = torch.randn(c.B * T, Hq * D, generator=g).to(dtype)
    for b in range(c.B):  # rows not in use may hold anything
        q.view(c.B, T, -1)[b, c.used(b):] = math.nan
    q = q.to(DEV)
    out, stats = attend(c, q, Hq)
    assert torch.equal(stats.view(c.B, T, -1)[2 % c.B, c.used(2 % c.B):], torch.full_like(stats.view(c.B, T, -1)[2 % c.B, c.used(2 % c.B):], 7.0))
    stats.view(c.B, T, -1)[[b for b in range(c.B) if not c.used(b)]] = math.nan
    keep = n_keep = None
    if paths is not None:
        keep = i32([p + [99] * (T - len(p)) for p in paths])
        n_keep = i32([len(p) for p in paths])
    room = max(max(lens), 0) + T + 2
    score = torch.rand(c.B, heads, room, generator=g)
    at = torch.randint(-9, 99999, (c.B * T,), generator=g, dtype=torch.int32)
    position = torch.full((c.B, heads, room), -5, dtype=torch.int32, device=DEV)
    start = score.to(DEV)
    other = torch.full_like(start, 7.0) if apart else None
    ws = qlin.new_workspace(256, DEV)
    got = qlin.kv_weigh(c.cache, c.step, q, stats, start, keep=keep, n_keep=n_keep, decay=0.75, score_out=other,
                        position_out=position, at=at.to(DEV) if apart else None, ws=ws)
    assert got is (other if apart else start) and qlin.read_device_status(ws) == 0
    if apart:
        assert torch.equal(start.cpu(), score)
    got, position = got.cpu(), position.cpu()
    for b, n in enumerate(lens):
        path = None if paths is None else paths[b]
        kept = (list(range(c.used(b))) if path is None else path) if n >= 0 else []
        end = max(n, 0) + len(kept)
        for h in range(heads):
            untouched = torch.full((room,), 7.0) if apart else score[b, h]
            assert torch.equal(got[b, h, end:], untouched[end:])
            if n < 0:
                continue
            want, bound = reference(c, q, stats, Hq, b, h, path)
            want[:n] += 0.75 * score[b, h, :n].double()
            bound[:n] += 2.0 ** -24 * want[:n]
            off = (got[b, h, :end].double() - want).abs()
            assert (off <= bound).all(), (b, h, float((off / bound).max()))
            expect = [int(at[b * T + r]) if apart else n + c.depth[r] for r in kept]
            assert position[b, h, max(n, 0):end].tolist() == expect
            assert (position[b, h, : max(n, 0)] == -5).all() and (position[b, h, end:] == -5).all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_statistics_are_the_softmax_ones(dtype):
    """2^r l is the sum of 2^x over what a row sees, and the weights of all tokens add up to the query heads."""
    c = Case([900, 3, 0], 4, 2, 128, 32, dtype, seed=2, parents=[-1, 0, 0, 2])
    q = torch.randn(12, 8 * 128, generator=torch.Generator().manual_seed(3)).to(dtype).to(DEV)
    plain = qlin.tree_attention(c.cache, c.step, q)
    out, stats = attend(c, q, 8)
    assert torch.equal(out.view(torch.int16), plain.view(torch.int16))
    for b in range(3):
        for h in range(2):
            qq = rows_of(c, q, b, h, 8)
            for t in range(4):
                seen = c.seen(b, t)
                x = qq[t] @ c.host[b][0][seen, h].double().T * (128 ** -0.5 * math.log2(math.e))
                st = stats.view(3, 4, 2, 4, 2)[b, t, h].cpu().double()
                assert ((torch.exp2(x - st[:, :1]).sum(1) / st[:, 1] - 1).abs() < 2e-5).all()
    score = torch.zeros(3, 2, 910, device=DEV)
    qlin.kv_weigh(c.cache, c.step, q, stats, score)
    assert ((score.sum(-1) - 16).abs() < 1e-3).all()


def test_keys_that_are_not_finite_reach_their_own_token_alone():
    """... and masked rows of the step reach nothing."""
    c = Case([200], 3, 1, 64, 16, BF, seed=2, parents=[-1, 0, 0])
    q = torch.randn(3, 4 * 64, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    _, stats = attend(c, q, 4)
    want = qlin.kv_weigh(c.cache, c.step, q, stats, torch.zeros(1, 1, 210, device=DEV)).clone()
    p, r = c.places(0, 17, 1)
    c.k[p, :, r] = math.nan
    p, r = c.places(0, 202, 1)
    c.k[p, :, r] = math.inf  # row 2, which rows 0 and 1 do not see
    got = qlin.kv_weigh(c.cache, c.step, q, stats, torch.zeros(1, 1, 210, device=DEV))
    assert got[0, 0, 17].isnan()
    same = [i for i in range(210) if i not in (17, 202)]
    assert torch.equal(got[0, 0, same], want[0, 0, same])
    path = qlin.kv_weigh(c.cache, c.step, q, stats, torch.zeros(1, 1, 210, device=DEV), keep=i32([[0, 1, 0]]), n_keep=i32([2]))
    assert path[0, 0, 202] == 0 and path[0, 0, :17].isfinite().all() and path[0, 0, 18:].isfinite().all()


def test_huge_scores_give_whole_weights():
    """Scores past fp32's unit steps: the largest takes all, equal ones share."""
    c = Case([300], 1, 1, 128, 32, BF, seed=2)
    k = c.host[0][0]
    k[:] = torch.rand(k.shape, generator=torch.Generator().manual_seed(5)).to(BF)
    k[5] = k[250] = 100.0
    c.put(0, 0, k, c.host[0][1])
    q = torch.full((1, 128), 2.0 ** 100, dtype=BF, device=DEV)
    _, stats = attend(c, q, 1)
    got = qlin.kv_weigh(c.cache, c.step, q, stats, torch.zeros(1, 1, 301, device=DEV)).cpu()[0, 0]
    want = torch.zeros(301)
    want[[5, 250]] = 0.5
    assert torch.equal(got, want)


def test_bad_lists_and_full_arrays_are_reported():
    c = Case([50, 60], 4, 2, 64, 16, BF, seed=2)
    q = torch.randn(8, 2 * 64, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    _, stats = attend(c, q, 2)
    for keep, n in (([[0, 2, 1, 3]] * 2, [3, 2]), ([[0, 1, 4, 0]] * 2, [3, 0]), ([[0, 1, 2, 3]] * 2, [5, 1]), ([[-1, 1, 2, 3]] * 2, [1, -2])):
        ws = qlin.new_workspace(256, DEV)
        score = torch.ones(2, 2, 70, device=DEV)
        got = qlin.kv_weigh(c.cache, c.step, q, stats, score, keep=i32(keep), n_keep=i32(n), decay=0.5, ws=ws)
        assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX
        assert (got[0, :, :50] == 0.5).all() and (got[0, :, 50:] == 1).all()
    ws = qlin.new_workspace(256, DEV)
    score = torch.ones(2, 2, 70, device=DEV)
    qlin.kv_weigh(c.cache, c.step, q, stats, score[:, :, :52], ws=ws)
    assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX and (score[:, :, 52:] == 1).all()
    whole = qlin.kv_weigh(c.cache, c.step, q, stats, torch.ones(2, 2, 70, device=DEV))
    assert torch.equal(score[:, :, :52], whole[:, :, :52])
    table = c.table.clone()
    table[1, 1] = 1 << 28
    step = qlin.KVStep(table.to(DEV), c.step.len, 4)
    ws = qlin.new_workspace(256, DEV)
    got = qlin.kv_weigh(c.cache, step, q, stats, torch.ones(2, 2, 70, device=DEV), ws=ws)
    assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX and torch.equal(got[0], whole[0])


@pytest.mark.parametrize("copy", [0, 1, 3])
def test_an_expired_wait_is_reported_not_hung(copy):
    c = Case([40000], 2, 1, 128, 64, BF, seed=2)
    q = torch.randn(2, 4 * 128, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    _, stats = attend(c, q, 4)
    ws = qlin.new_workspace(256, DEV)
    start = torch.rand(1, 1, 40002, device=DEV)
    want = qlin.kv_weigh(c.cache, c.step, q, stats, start.clone(), ws=ws)
    assert qlin.read_device_status(ws) == 0
    assert qlin.debug_kv_weigh_fault(c.cache, c.step, q, stats, start.clone(), ws, copy) == 0
    torch.cuda.synchronize()
    assert qlin.read_device_status(ws) == qlin.ERR_DEVICE_TIMEOUT
    ws = qlin.new_workspace(256, DEV)
    assert torch.equal(qlin.kv_weigh(c.cache, c.step, q, stats, start.clone(), ws=ws), want)
    assert qlin.read_device_status(ws) == 0


def test_many_sequences_replayed_with_other_lengths():
    """Captured behind attention, with programmatic launches; lengths, rows and scores change; another stream's eager call."""
    lens = [70 * (i % 11) + i for i in range(40)]
    c = Case(lens, 2, 2, 64, 16, FP, seed=4)
    q = torch.randn(80, 6 * 64, generator=torch.Generator().manual_seed(3)).half().to(DEV)
    stats, out = torch.empty(80, 6, 2, device=DEV), torch.empty(80, 6 * 64, dtype=BF, device=DEV)
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(c.cache, 40, 2, 6), DEV)
    score = torch.zeros(40, 2, 800, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        qlin.tree_attention(c.cache, c.step, q, out=out, ws=ws, stats=stats, flags=qlin.FLAG_PDL)
        qlin.kv_weigh(c.cache, c.step, q, stats, score, flags=qlin.FLAG_PDL, ws=ws)

    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for cut in (0, 1, 33):
        now = [max(0, n - cut) if cut != 33 or i % 3 else -1 for i, n in enumerate(lens)]
        c.step.len.copy_(i32(now))
        score.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        got = score.clone()
        score.fill_(1.0)
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        assert torch.equal(score, got)
        for b, n in enumerate(now):
            if n >= 0:
                assert ((got[b, :, : n + 2].sum(-1) - n - 6).abs() < 1e-3 * (n + 6)).all()
                assert (got[b, :, n + 2:] == 1).all()
            else:
                assert (got[b] == 1).all()


def test_append_attend_weigh_keep_evict_as_one_step():
    """The operators around a cache as a decoder uses them, in one captured step: the cache stays within its room, and what
    attention sees is what has stayed."""
    heads, Hq, D, T, room = 2, 4, 64, 3, 96
    c = Case([90], T, heads, D, 16, BF, seed=3, fill=False, parents=[-1, 0, 0])
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    k, v = torch.zeros(8, heads, 16, D, dtype=BF, device=DEV), torch.zeros(8, heads, 16, D, dtype=BF, device=DEV)
    length = i32([0])
    cache = qlin.KVCache(k, v)
    step = qlin.KVStep(table, length, T, depth=i32([0, 1, 1]), mask=i32([1, 3, 5]))
    g = torch.Generator(device=DEV).manual_seed(4)
    q, nk, nv = (torch.empty(T, h * D, device=DEV) for h in (Hq, heads, heads))
    at, keep, n_keep, most, since = i32([0, 0, 0]), i32([[0, 2, 0]]), i32([2]), i32([room]), i32([0])
    turns = qlin.rope_turns(1e4, D, device=DEV)
    q_out, out = torch.empty(T, Hq * D, dtype=BF, device=DEV), torch.empty(T, Hq * D, dtype=BF, device=DEV)
    stats = torch.empty(T, Hq, 2, device=DEV)
    score, position = torch.zeros(1, heads, room + T, device=DEV), torch.full((1, heads, room + T), -1, dtype=torch.int32, device=DEV)
    ws = qlin.new_workspace(qlin.tree_attention_workspace_bytes(cache, 1, T, Hq), DEV)
    we = qlin.new_workspace(qlin.kv_evict_workspace_bytes(cache, step, room + T), DEV)

    def call(flags=qlin.FLAG_PDL):
        qlin.kv_append(cache, step, q, nk, nv, turns=turns, position=at, q_out=q_out, ws=ws, flags=flags)
        qlin.tree_attention(cache, step, q_out, out=out, ws=ws, stats=stats, flags=flags)
        qlin.kv_weigh(cache, step, q_out, stats, score, keep=keep, n_keep=n_keep, position_out=position, at=at, ws=ws, flags=flags)
        qlin.kv_keep(cache, step, keep, n_keep, len_out=length, ws=ws, flags=flags)
        qlin.kv_evict(cache, step, score, most, since=since, position=position, len_out=length, ws=we, flags=flags)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    host = {}  # position: k, v of each head
    now = 0
    for i in range(80):
        for x in (q, nk, nv):
            x.copy_(torch.randn(x.shape, device=DEV, generator=g))
        at.copy_(i32([now, now + 1, now + 1]))
        since.fill_(now - 8)
        if i % 2:
            call(0)
        else:
            graph.replay()
        for row, p in ((0, now), (2, now + 1)):
            host[p] = (R.append_row(nk[row].cpu().view(heads, D), None, 1e-6, p, [1e4 ** (-2.0 * j / D) for j in range(D // 2)], False),
                       nv[row].cpu().view(heads, D).double())
        now += 2
        n = min(now, room)
        assert length.tolist() == [n]
        if i % 16 == 15:
            assert qlin.read_device_status(ws) == 0 and qlin.read_device_status(we) == 0
            kk, vv = (x[table[0].long()].transpose(0, 1).reshape(heads, -1, D)[:, :n].cpu().double() for x in (k, v))
            for h in range(heads):
                places = position[0, h, :n].tolist()
                assert len(set(places)) == n and set(range(now - 8, now)) <= set(places)
                for j, p in enumerate(places):
                    assert ((kk[h, j] - host[p][0][h]).abs() <= R.append_bound(host[p][0], BF)[h]).all()
                    assert ((vv[h, j] - host[p][1][h]).abs() <= 2.0 ** -8 * host[p][1][h].abs()).all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_statistics_do_not_depend_on_what_shared_memory_held(dtype):
    """The same call behind one that leaves large numbers where rows of a fuller step lie: the same bits."""
    c = Case([300], 4, 4, 128, 64, dtype, seed=3)
    g = torch.Generator().manual_seed(9)
    q = torch.randn(4, 8 * 128, generator=g).to(dtype).to(DEV)
    full = Case([300], 16, 4, 128, 64, dtype, seed=4)
    large = (torch.randn(16, 8 * 128, generator=g) * 2.0 ** 14).to(dtype).to(DEV)
    small = torch.zeros_like(large)
    results = []
    for before in (small, large, small):
        qlin.tree_attention(full.cache, full.step, before, scale=1e4)
        results.append(attend(c, q, 8))
    for out, stats in results[1:]:
        assert torch.equal(stats, results[0][1]) and torch.equal(out.view(torch.int16), results[0][0].view(torch.int16))


def test_arguments_of_the_two_ways_agree():
    """The same operands as plain tensors (read by the extension) and as slices of wider ones (read one by one)."""
    c = Case([500, 77], 3, 2, 64, 16, BF, seed=5, parents=[-1, 0, 0])
    g = torch.Generator().manual_seed(6)
    q = torch.randn(6, 4 * 64, generator=g).bfloat16().to(DEV)
    _, stats = attend(c, q, 4)
    keep, n_keep, score = i32([[0, 2, 0], [0, 1, 0]]), i32([2, 1]), torch.rand(2, 2, 520, generator=g).to(DEV)
    position = torch.zeros(2, 2, 520, dtype=torch.int32, device=DEV)
    plain = qlin.kv_weigh(c.cache, c.step, q, stats, score, keep=keep, n_keep=n_keep, score_out=torch.zeros_like(score), position_out=position)
    wide_q = torch.zeros(6, 4 * 64 + 16, dtype=BF, device=DEV)
    wide_q[:, 8:-8] = q
    wide = torch.zeros(2, 2, 2, 530, device=DEV)
    wide[:, 0, :, 5:525] = score
    wide_keep = torch.zeros(2, 9, dtype=torch.int32, device=DEV)
    wide_keep[:, 4:7] = keep
    out = torch.zeros(2, 2, 600, device=DEV)[:, :, 3:523]
    where = torch.zeros(2, 2, 600, dtype=torch.int32, device=DEV)[:, :, 3:523]
    got = qlin.kv_weigh(c.cache, c.step, wide_q[:, 8:-8], stats, wide[:, 0, :, 5:525], keep=wide_keep[:, 4:7], n_keep=n_keep, score_out=out,
                        position_out=where)
    assert torch.equal(got, plain) and torch.equal(where, position)
    with pytest.raises(ValueError, match="strides"):
        qlin.kv_weigh(c.cache, c.step, q, stats, score, score_out=out, position_out=position)
    with pytest.raises(ValueError, match="stats"):
        qlin.kv_weigh(c.cache, c.step, q, stats[:, :2], score)
    with pytest.raises(ValueError, match="n_keep"):
        qlin.kv_weigh(c.cache, c.step, q, stats, score, keep=keep, n_keep=n_keep[:1])
    with pytest.raises(qlin.QlinError):
        qlin.kv_weigh(c.cache, c.step, q, stats, score, n_keep=n_keep)
    with pytest.raises(qlin.QlinError):
        qlin.kv_weigh(c.cache, c.step, q, stats, score, decay=math.nan)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("poison", [math.nan, math.inf])
@pytest.mark.parametrize("place", [17, 202])  # a committed token; row 2's own, which rows 0 and 1 do not see
def test_a_key_that_is_not_finite_before_attention(dtype, poison, place):
    """Rows whose softmax has become NaN by it weigh nothing in that cache head; what other rows and heads give is what it was,
    and what stays by the scores stays."""
    c = Case([200], 3, 2, 64, 16, dtype, seed=2, parents=[-1, 0, 0])
    q = torch.randn(3, 4 * 64, generator=torch.Generator().manual_seed(3)).to(dtype).to(DEV)
    start = torch.rand(1, 2, 203, generator=torch.Generator().manual_seed(4)).to(DEV)
    _, stats = attend(c, q, 4)
    want = qlin.kv_weigh(c.cache, c.step, q, stats, start, score_out=torch.zeros_like(start), decay=0.5)
    without = qlin.kv_weigh(c.cache, c.step, q, stats, start, score_out=torch.zeros_like(start), decay=0.5, keep=i32([[0, 1, 0]]),
                            n_keep=i32([2]))
    p, r = c.places(0, place, 1)
    c.k[p, 0, r] = poison  # infinities of both signs in the products: NaN
    _, stats = attend(c, q, 4)
    assert not stats.view(3, 2, 2, 2)[2, 0, :, 1].isfinite().any()
    got = qlin.kv_weigh(c.cache, c.step, q, stats, start, score_out=torch.zeros_like(start), decay=0.5)
    assert torch.equal(got[0, 1], want[0, 1])
    others = [i for i in range(203) if i != place]
    if place == 17:  # no row of the head weighs anything
        assert torch.equal(got[0, 0, :200][others[:199]], 0.5 * start[0, 0, :200][others[:199]]) and (got[0, 0, 200:] == 0).all()
    else:
        assert torch.equal(got[0, 0, others], without[0, 0, others])
    c.step.len.fill_(203)
    best = got[0].nan_to_num(nan=-1.0).topk(60, -1).values.sort(-1).values
    qlin.kv_evict(c.cache, c.step, got, i32([60]))
    assert torch.equal(got[0, :, :60].sort(-1).values, best)


def test_a_query_row_that_is_not_finite():
    """It weighs nothing; the other rows weigh what they did."""
    c = Case([300], 3, 2, 128, 32, BF, seed=2, parents=[-1, 0, 0])
    q = torch.randn(3, 4 * 128, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    _, stats = attend(c, q, 4)
    without = qlin.kv_weigh(c.cache, c.step, q, stats, torch.zeros(1, 2, 303, device=DEV), keep=i32([[0, 2, 0]]), n_keep=i32([2]))
    q[1] = math.nan
    _, stats = attend(c, q, 4)
    got = qlin.kv_weigh(c.cache, c.step, q, stats, torch.zeros(1, 2, 303, device=DEV))
    assert torch.equal(got[:, :, :301], without[:, :, :301]) and (got[:, :, 301] == 0).all()
    assert torch.equal(got[:, :, 302], without[:, :, 301])


@pytest.mark.parametrize("apart", [False, True], ids=["in place", "apart"])
def test_tokens_on_a_page_out_of_range_are_left_as_they_were(apart):
    """Committed ones, and a step's own; the others of the sequence get what they got."""
    c = Case([50, 60], 4, 2, 64, 16, BF, seed=2)
    q = torch.randn(8, 2 * 64, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    _, stats = attend(c, q, 2)
    start = torch.rand(2, 2, 70, generator=torch.Generator().manual_seed(4)).to(DEV)
    want = qlin.kv_weigh(c.cache, c.step, q, stats, start, score_out=torch.zeros_like(start), decay=0.5)
    table = c.table.clone()
    table[0, 3], table[1, 1] = -1, 1 << 28
    step = qlin.KVStep(table.to(DEV), c.step.len, 4, depth=c.step.depth, mask=c.step.mask)
    out, ws = torch.full_like(start, 7.0) if apart else start.clone(), qlin.new_workspace(256, DEV)
    before = out.clone()
    position = torch.full((2, 2, 70), -5, dtype=torch.int32, device=DEV)
    qlin.kv_weigh(c.cache, step, q, stats, start if apart else out, score_out=out, position_out=position, decay=0.5, ws=ws)
    assert qlin.read_device_status(ws) == qlin.ERR_BAD_INDEX
    lost = torch.zeros(2, 2, 70, dtype=torch.bool, device=DEV)
    lost[0, :, 48:] = lost[1, :, 16:32] = lost[1, :, 64:] = True
    assert torch.equal(out[lost], before[lost]) and torch.equal(out[~lost], want[~lost])
    assert (position[0] == -5).all() and (position[1, :, :60] == -5).all() and position[1, 0, 60:64].tolist() == [60, 61, 62, 63]


def test_tokens_behind_the_table_are_reported():
    """Committed ones, and kept rows' own; rows that are not kept may lie behind it."""
    for lens, keep, status in (([50, 60], None, 0), ([50, 61], None, qlin.ERR_BAD_INDEX), ([64, 64], [], 0), ([63, 60], [0], 0),
                               ([63, 62], [0, 2], qlin.ERR_BAD_INDEX), ([62, 3], [1], 0), ([50, 70], [], qlin.ERR_BAD_INDEX),
                               ([200, -1], [0], qlin.ERR_BAD_INDEX), ([-1, 0], [0, 1, 2, 3], 0)):
        c = Case(lens, 4, 2, 64, 16, BF, seed=2)
        q = torch.randn(8, 2 * 64, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
        _, stats = attend(c, q, 2)
        lists = {} if keep is None else dict(keep=i32([keep + [0] * (4 - len(keep))] * 2), n_keep=i32([len(keep)] * 2))
        start = torch.rand(2, 2, 210, generator=torch.Generator().manual_seed(4)).to(DEV)
        want = qlin.kv_weigh(c.cache, c.step, q, stats, start, score_out=start.clone(), decay=0.5, **lists)
        step = qlin.KVStep(c.table[:, :4].to(DEV), c.step.len, 4)
        ws = qlin.new_workspace(256, DEV)
        got = qlin.kv_weigh(c.cache, step, q, stats, start, score_out=start.clone(), decay=0.5, ws=ws, **lists)
        assert qlin.read_device_status(ws) == status, (lens, keep)
        for b, n in enumerate(lens):
            kept = [r for r in (range(4) if keep is None else keep) if n >= 0 and n + r < 64]
            end = min(max(n, 0) + len(kept), 64)
            assert torch.equal(got[b, :, :end], want[b, :, :end]) and torch.equal(got[b, :, max(end, 64):], start[b, :, max(end, 64):])


@pytest.mark.parametrize("copy", [9, 13, 26])
def test_a_wait_that_expires_far_into_a_run(copy):
    """Behind the ring's first round and the accumulators' first use."""
    n = 152 * 128 * 16
    c = Case([n], 2, 1, 128, 256, BF, seed=2)
    q = torch.randn(2, 4 * 128, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    _, stats = attend(c, q, 4)
    ws = qlin.new_workspace(256, DEV)
    start = torch.rand(1, 1, n + 2, device=DEV)
    want = qlin.kv_weigh(c.cache, c.step, q, stats, start.clone(), ws=ws)
    assert qlin.debug_kv_weigh_fault(c.cache, c.step, q, stats, start.clone(), ws, copy) == 0
    torch.cuda.synchronize()
    assert qlin.read_device_status(ws) == qlin.ERR_DEVICE_TIMEOUT
    ws = qlin.new_workspace(256, DEV)
    assert torch.equal(qlin.kv_weigh(c.cache, c.step, q, stats, start.clone(), ws=ws), want)
    assert qlin.read_device_status(ws) == 0
