"""Appending at positions, weighing, eviction and adjusted logits on the host: what they refuse before anything reaches
the GPU, and empty calls."""
import ctypes

import pytest
import torch

import __graft_entry__
from test_step_host import BAD_CACHE, BAD_STEP, cache, step
from w6a8_quantized_linear_gb300 import qlin


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return qlin.lib()


def append_at(L, c=None, s=None, **kw):
    a = dict(Hq=8, src=2, q=1 << 20, qs=1024, k=4096, ks=512, v=4096, vs=512, nt=8, turns=4096, position=1 << 16, ps=3, axes=3,
             axis=bytes([0, 1, 2, 0, 1, 2, 0, 1]), qo=1 << 24, qos=1024, flags=0)
    a.update(kw)
    c, s = c or cache(), s or step()
    return L.qlin_kv_append_at(ctypes.addressof(c), ctypes.addressof(s), a["Hq"], a["src"], a["q"], a["qs"], a["k"], a["ks"],
                               a["v"], a["vs"], None, None, 1e-6, a["turns"], a["nt"], 0, a["position"], a["ps"], a["axes"],
                               a["axis"], a["qo"], a["qos"], None, 0, a["flags"], None)


@pytest.mark.parametrize("bad", [dict(position=None), dict(position=4098), dict(ps=2), dict(axes=0), dict(axes=5, ps=5), dict(axis=None),
                                 dict(axis=bytes([0, 1, 2, 3, 0, 0, 0, 0])), dict(axes=1, ps=0), dict(nt=65), dict(flags=2),
                                 dict(qo=1 << 16), dict(qo=(1 << 16) + 16, qos=1024)])
def test_append_at_refusals(L, bad):
    assert append_at(L, **bad) == qlin.ERR_INVALID_ARG


def test_append_at_refuses_what_append_does(L):
    for kw, status in BAD_CACHE:
        assert append_at(L, c=cache(**kw)) == status
    for kw, status in BAD_STEP:
        assert append_at(L, s=step(**kw)) == status
    assert append_at(L, s=step(B=0), position=None) == qlin.OK
    assert append_at(L, s=step(T=0), position=None, q=None, k=None, v=None) == qlin.OK


def test_rope_axes():
    assert qlin.rope_axes((2, 1, 1)) == bytes([0, 0, 1, 2])
    assert qlin.rope_axes((3, 1, 2), dealt=True) == bytes([0, 1, 2, 0, 2, 0])
    assert qlin.rope_axes((0, 2), dealt=True) == bytes([1, 1]) and qlin.rope_axes((0,)) == b""
    for bad in ((), (1, 2, 3, 4, 5), (1, -1)):
        with pytest.raises(ValueError):
            qlin.rope_axes(bad)


def test_the_binding_refuses_positions_on_the_cpu():
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    s = qlin.KVStep(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="CPU"):
        qlin.kv_append(qlin.KVCache(k, k), s, q=torch.zeros(2, 64), position=torch.zeros(2, dtype=torch.int32))


def adjust(so, /, B=2, T=3, V=1000, dtype=2, logits=1 << 20, ld=1000, out=1 << 24, old=1000, flags=0, struct=True, **kw):
    a = dict(history=4096, history_len=None, prompt_len=None, draft=4096, mask=None, repetition=4096, presence=None, frequency=None,
             bias_token=4096, bias=4096, allowed=4096, history_stride=50, tree_stride=0, bias_stride=0, allowed_stride=32, L=50, n_bias=9)
    a.update(kw)
    s = qlin._ADJUSTMENTS.pack(*[a[n] or 0 for n in (
        "history", "history_len", "prompt_len", "draft", "mask", "repetition", "presence", "frequency", "bias_token", "bias",
        "allowed", "history_stride", "tree_stride", "bias_stride", "allowed_stride", "L", "n_bias")])
    return so.qlin_adjust_logits(B, T, V, dtype, logits, ld, out, old, s if struct else None, flags, None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(V=0), dict(dtype=1), dict(dtype=3), dict(logits=None), dict(out=None), dict(ld=999), dict(old=999),
    dict(logits=(1 << 20) + 2), dict(out=(1 << 24) + 1, dtype=0), dict(flags=2), dict(struct=False), dict(history=None),
    dict(history=4097), dict(history_stride=49), dict(L=-1), dict(n_bias=-1), dict(bias=None), dict(bias_token=None),
    dict(bias_stride=8), dict(bias_stride=-1), dict(tree_stride=2), dict(tree_stride=-3), dict(allowed_stride=31),
    dict(allowed_stride=-1), dict(allowed=4098), dict(out=(1 << 20) + 4), dict(out=1 << 20, old=1001),
    dict(out=(1 << 20) - 4000 * 6 + 4), dict(draft=4098), dict(repetition=4098)])
def test_adjust_refusals(L, bad):
    assert adjust(L, **bad) == qlin.ERR_INVALID_ARG


def test_adjust_limits_and_empty_calls(L):
    for bad in (dict(V=524289, ld=524289, old=524289), dict(T=33), dict(L=1000001, history_stride=1000001), dict(n_bias=1025),
                dict(B=65536), dict(B=65535, T=257, draft=None)):
        assert adjust(L, **bad) == qlin.ERR_UNSUPPORTED
    assert adjust(L, B=0, logits=None, out=None) == qlin.OK
    assert adjust(L, T=0, logits=None, out=None) == qlin.OK


def test_the_binding_refuses_adjustments_it_can_see():
    x = torch.zeros(4, 10)
    with pytest.raises(ValueError, match="CPU"):
        qlin.adjust_logits(x)
    with pytest.raises(ValueError, match="contiguous"):
        qlin.adjust_logits(torch.zeros(10, 4).t())


def evict(so, /, c=None, s=None, **kw):
    a = dict(score=1 << 20, position=None, ss=4 * 64, hs=64, score_out=1 << 20, position_out=None, oss=4 * 64, ohs=64, room=64,
             n_keep=4096, first=0, since=None, len_out=None, ws=1 << 30, wsb=1 << 20, flags=0)
    a.update(kw)
    c, s = c or cache(), s or step()
    return so.qlin_kv_evict(ctypes.addressof(c), ctypes.addressof(s), *[a[n] for n in (
        "score", "position", "ss", "hs", "score_out", "position_out", "oss", "ohs", "room", "n_keep", "first", "since", "len_out",
        "ws", "wsb", "flags")], None)


@pytest.mark.parametrize("bad", [
    dict(score=None), dict(score_out=None), dict(n_keep=None), dict(ws=None), dict(ws=4096 + 16), dict(room=-1), dict(first=-1),
    dict(score=4098), dict(position=4097), dict(since=4098), dict(len_out=4097), dict(n_keep=4098), dict(flags=2), dict(hs=63),
    dict(ss=64), dict(ohs=63), dict(oss=64), dict(ss=-256), dict(score_out=(1 << 20) + 4), dict(score_out=(1 << 20) - 2048 + 4),
    dict(oss=5 * 64), dict(position=1 << 20), dict(position_out=1 << 20), dict(position=1 << 24, position_out=(1 << 24) + 64),
    dict(position=1 << 24, score_out=1 << 24), dict(score_out=1 << 24, position_out=(1 << 24) + 1024)])
def test_evict_refusals(L, bad):
    assert evict(L, **bad) == qlin.ERR_INVALID_ARG


def test_evict_refuses_what_others_do_and_limits(L):
    for kw, status in BAD_CACHE:
        assert evict(L, c=cache(**kw)) == status
    for kw, status in BAD_STEP:
        assert evict(L, s=step(**kw)) == status
    assert evict(L, wsb=256) == qlin.ERR_WORKSPACE
    assert evict(L, room=1 << 21, hs=1 << 21, ss=1 << 23, ohs=1 << 21, oss=1 << 23) == qlin.ERR_UNSUPPORTED
    assert evict(L, s=step(B=1 << 19), ss=64, hs=1 << 26) == qlin.ERR_UNSUPPORTED
    assert evict(L, s=step(B=0), score=None, ws=None) == qlin.OK
    n = ctypes.c_size_t()
    c = cache()
    assert L.qlin_kv_evict_workspace_bytes(ctypes.addressof(c), 2, 64, ctypes.byref(n)) == qlin.OK
    assert n.value >= 256 + 8 * 8 + 8 * 2 * 32 * 4
    assert L.qlin_kv_evict_workspace_bytes(ctypes.addressof(c), -1, 64, ctypes.byref(n)) == qlin.ERR_INVALID_ARG
    assert L.qlin_kv_evict_workspace_bytes(ctypes.addressof(c), 2, 64, None) == qlin.ERR_INVALID_ARG


def weigh(so, /, c=None, s=None, **kw):
    a = dict(Hq=8, q=4096, qs=1024, stats=4096, scale=0.1, keep=None, ks=0, n_keep=None, decay=1.0, score=1 << 20, ss=256, hs=64,
             score_out=1 << 20, position_out=None, oss=256, ohs=64, room=64, at=None, ws=None, wsb=0, flags=0)
    a.update(kw)
    c, s = c or cache(), s or step()
    return so.qlin_kv_weigh(ctypes.addressof(c), ctypes.addressof(s), *[a[n] for n in (
        "Hq", "q", "qs", "stats", "scale", "keep", "ks", "n_keep", "decay", "score", "ss", "hs", "score_out", "position_out", "oss",
        "ohs", "room", "at", "ws", "wsb", "flags")], None)


@pytest.mark.parametrize("bad", [
    dict(Hq=0), dict(Hq=6), dict(q=None), dict(q=4104), dict(qs=1023), dict(stats=None), dict(stats=4100), dict(scale=float("inf")),
    dict(decay=float("nan")), dict(keep=4096, ks=3), dict(n_keep=4096), dict(keep=4096, n_keep=4096, ks=2), dict(keep=4097, n_keep=4096, ks=3),
    dict(score=None), dict(score_out=None), dict(score=4098), dict(room=-1), dict(hs=63), dict(oss=64), dict(score_out=(1 << 20) + 8),
    dict(oss=512), dict(position_out=1 << 20), dict(at=4098), dict(ws=4096 + 8, wsb=256), dict(flags=4),
    dict(score_out=1 << 24, q=(1 << 24) + 1024), dict(position_out=1 << 24, stats=(1 << 24) + 8), dict(score_out=1 << 24, at=(1 << 24) + 2040)])
def test_weigh_refusals(L, bad):
    assert weigh(L, **bad) == qlin.ERR_INVALID_ARG


def test_weigh_refuses_what_others_do_and_limits(L):
    for kw, status in BAD_CACHE:
        assert weigh(L, c=cache(**kw)) == status
    for kw, status in BAD_STEP:
        assert weigh(L, s=step(**kw)) == status
    assert weigh(L, s=step(T=33)) == qlin.ERR_UNSUPPORTED
    assert weigh(L, Hq=4 * 43, qs=4 * 43 * 128) == qlin.ERR_UNSUPPORTED
    assert weigh(L, room=1 << 21) == qlin.ERR_UNSUPPORTED
    assert weigh(L, ws=4096, wsb=255) == qlin.ERR_WORKSPACE
    assert weigh(L, s=step(B=0), q=None, stats=None, score=None) == qlin.OK
    c, s = cache(), step()
    fault = lambda c, copy: L.qlin_debug_kv_weigh_fault(  # noqa: E731
        ctypes.addressof(c), ctypes.addressof(s), 8, 4096, 1024, 4096, 0.1, 1 << 20, 256, 64, 1 << 20, 64, None, 0, copy, None)
    assert fault(c, -1) == qlin.ERR_INVALID_ARG and fault(cache(dtype=1), 0) == qlin.ERR_UNSUPPORTED


def test_attention_statistics_refusals(L):
    c, s = cache(), step()
    call = lambda stats, q=1 << 24, s=s: L.qlin_tree_attention_stats(  # noqa: E731
        ctypes.addressof(c), ctypes.addressof(s), 8, q, 1024, 0.1, 1 << 28, 1024, stats, 1 << 32, 1 << 30, 0, None)
    for bad in (None, 4100, 1 << 24, (1 << 28) + 64):
        assert call(bad) == qlin.ERR_INVALID_ARG
    assert call(None, s=step(T=0)) == qlin.OK
