"""The step operators (append, tree attention, keep, sample) on the host: what
they refuse before anything reaches the GPU, empty calls, and the rotation
frequencies."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import __graft_entry__
from w6a8_quantized_linear_gb300 import qlin


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return qlin.lib()


def cache(**kw):
    """A cache struct whose addresses are never followed."""
    a = dict(k=4096, v=8192, pages=10, page_stride=4 * 16 * 128, head_stride=16 * 128, token_stride=128, dtype=0, heads=4,
             width=128, page_size=16)
    a.update(kw)
    return qlin._CacheStruct(**a)


def step(**kw):
    a = dict(page_table=4096, len=4096, count=None, depth=None, mask=None, table_stride=5, tree_stride=0, B=2, T=3, max_pages=5)
    a.update(kw)
    return qlin._StepStruct(**a)


BAD_CACHE = [
    (dict(k=None), qlin.ERR_INVALID_ARG), (dict(v=4104), qlin.ERR_INVALID_ARG), (dict(dtype=2), qlin.ERR_INVALID_ARG),
    (dict(dtype=-1), qlin.ERR_INVALID_ARG), (dict(heads=0), qlin.ERR_INVALID_ARG), (dict(pages=0), qlin.ERR_INVALID_ARG),
    (dict(pages=1 << 31), qlin.ERR_INVALID_ARG), (dict(width=96), qlin.ERR_UNSUPPORTED), (dict(width=512), qlin.ERR_UNSUPPORTED),
    (dict(page_size=8), qlin.ERR_UNSUPPORTED), (dict(page_size=48), qlin.ERR_UNSUPPORTED), (dict(page_size=512), qlin.ERR_UNSUPPORTED),
    (dict(page_size=0), qlin.ERR_UNSUPPORTED), (dict(token_stride=120), qlin.ERR_INVALID_ARG),
    (dict(token_stride=132), qlin.ERR_INVALID_ARG), (dict(head_stride=0), qlin.ERR_INVALID_ARG),
    (dict(page_stride=-8), qlin.ERR_INVALID_ARG), (dict(page_stride=(1 << 36) + 8), qlin.ERR_INVALID_ARG),
]
BAD_STEP = [
    (dict(B=-1), qlin.ERR_INVALID_ARG), (dict(T=-1), qlin.ERR_INVALID_ARG), (dict(page_table=None), qlin.ERR_INVALID_ARG),
    (dict(len=None), qlin.ERR_INVALID_ARG), (dict(len=4098), qlin.ERR_INVALID_ARG), (dict(max_pages=0), qlin.ERR_INVALID_ARG),
    (dict(table_stride=4), qlin.ERR_INVALID_ARG), (dict(count=2), qlin.ERR_INVALID_ARG), (dict(mask=2), qlin.ERR_INVALID_ARG),
    (dict(depth=2), qlin.ERR_INVALID_ARG), (dict(tree_stride=2), qlin.ERR_INVALID_ARG), (dict(tree_stride=-3), qlin.ERR_INVALID_ARG),
]


def append(L, c=None, s=None, **kw):
    a = dict(Hq=8, src=2, q=4096, qs=1024, k=4096, ks=512, v=4096, vs=512, qg=None, kg=None, eps=1e-6, turns=None, nt=0, pairs=0,
             qo=4096, qos=1024, ws=None, wsb=0, flags=0)
    a.update(kw)
    c, s = c or cache(), s or step()
    return L.qlin_kv_append(ctypes.addressof(c), ctypes.addressof(s), a["Hq"], a["src"], a["q"], a["qs"], a["k"], a["ks"], a["v"],
                            a["vs"], a["qg"], a["kg"], a["eps"], a["turns"], a["nt"], a["pairs"], a["qo"], a["qos"], a["ws"],
                            a["wsb"], a["flags"], None)


def attention(L, c=None, s=None, **kw):
    a = dict(Hq=8, q=4096, qs=1024, scale=0.1, out=4096, os=1024, ws=4096, wsb=1 << 30, flags=0)
    a.update(kw)
    c, s = c or cache(), s or step()
    return L.qlin_tree_attention(ctypes.addressof(c), ctypes.addressof(s), a["Hq"], a["q"], a["qs"], a["scale"], a["out"], a["os"],
                                 a["ws"], a["wsb"], a["flags"], None)


def keep(L, c=None, s=None, **kw):
    a = dict(keep=4096, ks=3, n=4096, lo=4096, ws=None, wsb=0, flags=0)
    a.update(kw)
    c, s = c or cache(), s or step()
    return L.qlin_kv_keep(ctypes.addressof(c), ctypes.addressof(s), a["keep"], a["ks"], a["n"], a["lo"], a["ws"], a["wsb"],
                          a["flags"], None)


@pytest.mark.parametrize("call", [append, attention, keep])
def test_bad_caches_and_steps_are_refused(L, call):
    for kw, want in BAD_CACHE:
        assert call(L, c=cache(**kw)) == want, kw
    for kw, want in BAD_STEP:
        assert call(L, s=step(**kw)) == want, kw
    # no sequences or no rows: nothing is read, nothing enqueued
    assert call(L, s=step(B=0, page_table=None, len=None)) == qlin.OK
    assert call(L, s=step(T=0, page_table=None, len=None)) == qlin.OK
    assert call(L, flags=2) == qlin.ERR_INVALID_ARG


def test_append_refusals(L):
    bad = qlin.ERR_INVALID_ARG
    for kw in (dict(src=1), dict(src=3), dict(Hq=-1), dict(Hq=0), dict(q=4100), dict(qs=1023), dict(qs=1026), dict(qs=1016),
               dict(k=None), dict(v=None), dict(k=4104), dict(ks=508), dict(vs=514), dict(qo=None), dict(qo=4104), dict(qos=1020),
               dict(qg=8), dict(kg=4), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(nt=-1), dict(nt=65),
               dict(nt=64), dict(nt=64, turns=4), dict(pairs=2), dict(ws=128, wsb=256)):
        assert append(L, **kw) == bad, kw
    assert append(L, ws=256, wsb=255) == qlin.ERR_WORKSPACE
    assert append(L, Hq=16385, qs=16385 * 128, qos=16385 * 128) == qlin.ERR_UNSUPPORTED
    assert append(L, q=None, k=None, v=None) == qlin.OK  # nothing to do
    # rows beyond 2^31 - 1 do not fit a launch
    assert append(L, s=step(B=1 << 16, T=1 << 15)) == qlin.ERR_UNSUPPORTED


def test_attention_refusals(L):
    bad = qlin.ERR_INVALID_ARG
    for kw in (dict(Hq=0), dict(Hq=-4), dict(Hq=6), dict(q=None), dict(q=4104), dict(qs=1016), dict(qs=1028), dict(out=None),
               dict(out=4104), dict(os=1012), dict(scale=math.nan), dict(scale=math.inf), dict(ws=None), dict(ws=128)):
        assert attention(L, **kw) == bad, kw
    assert attention(L, s=step(T=33)) == qlin.ERR_UNSUPPORTED
    assert attention(L, s=step(T=32), Hq=20) == qlin.ERR_UNSUPPORTED  # 160 query rows per cache head
    assert attention(L, wsb=0) == qlin.ERR_WORKSPACE
    n = ctypes.c_size_t()
    c = cache()
    assert L.qlin_tree_attention_workspace_bytes(ctypes.addressof(c), 2, 3, 8, ctypes.byref(n)) == qlin.OK
    assert n.value >= 256
    assert attention(L, wsb=n.value - 1) == qlin.ERR_WORKSPACE
    assert L.qlin_tree_attention_workspace_bytes(ctypes.addressof(c), 2, 3, 8, None) == bad
    assert L.qlin_tree_attention_workspace_bytes(ctypes.addressof(c), -1, 3, 8, ctypes.byref(n)) == bad
    assert L.qlin_tree_attention_workspace_bytes(None, 2, 3, 8, ctypes.byref(n)) == bad


def test_attention_fault_export_refusals(L):
    def call(c=None, s=None, Hq=8, copy=0, ws=4096):
        c, s = c or cache(), s or step()
        return L.qlin_debug_tree_attention_fault(ctypes.addressof(c), ctypes.addressof(s), Hq, 4096, 1024, 0.1, 4096, 1024, ws,
                                                 1 << 30, copy, None)

    assert call(copy=-1) == qlin.ERR_INVALID_ARG
    assert call(ws=None) == qlin.ERR_INVALID_ARG
    assert call(c=cache(dtype=1)) == qlin.ERR_UNSUPPORTED
    assert call(c=cache(width=64)) == qlin.ERR_UNSUPPORTED
    assert call(s=step(T=17)) == qlin.ERR_UNSUPPORTED  # 34 query rows per cache head
    assert call(s=step(T=0)) == qlin.OK


def test_outputs_that_share_memory_with_inputs_are_refused(L):
    """Two rows of 1024 and 512 elements here (B = 2, T = 1): inside one another, end to end, and woven into one pool."""
    s = step(T=1)

    def att(q, qs, out, os):
        return attention(L, s=s, q=q, qs=qs, out=out, os=os)

    bad = qlin.ERR_INVALID_ARG
    M = 1 << 20
    for q, qs, out, os in ((M, 1024, M, 1024), (M, 1024, M + 16, 1024), (M, 1024, M + 4096 - 16, 1024), (M + 4096 - 16, 1024, M, 1024),
                           (M, 2048, M + 2048 - 16, 2048), (M, 2048, M + 4096 + 2048 - 16, 2048), (M, 2048, M, 4096),
                           (M, 4096, M + 4096, 1024)):
        assert att(q, qs, out, os) == bad, (q - M, qs, out - M, os)
    # apart: this far the arguments are right, and the call goes on to ask for a device
    for q, qs, out, os in ((M, 1024, M + 4096, 1024), (M + 4096, 1024, M, 1024), (M, 2048, M + 2048, 2048), (M + 2048, 2048, M, 2048),
                           (M, 1 << 40, M + 2048, 1 << 40), (M, 2048, M + 8192, 4096)):
        assert att(q, qs, out, os) != bad, (q - M, qs, out - M, os)

    def app(**kw):
        return append(L, s=s, **{**dict(src=0, q=M, qs=1024, k=2 * M, ks=512, v=3 * M, vs=512, qo=4 * M, qos=1024), **kw})

    assert app() != bad and app(src=2, qs=1024) != bad
    assert app(qo=M) != bad  # bf16 rows in their own places
    for kw in (dict(qo=M + 16), dict(qo=M, src=2), dict(qo=M, qos=1032), dict(qo=2 * M), dict(qo=2 * M + 2048 - 16), dict(qo=3 * M - 2048),
               dict(qo=3 * M + 1024 * 2 - 16)):
        assert app(**kw) == bad, kw
    # q, k and v woven into one projection of 2048 elements a row, q in its own place, or written between
    row = dict(qs=2048, k=M + 2048, ks=2048, v=M + 3072, vs=2048)
    assert app(**row, qo=M, qos=2048) != bad
    assert app(**row, qo=M + 2048, qos=2048) == bad and app(**row, qo=M + 16, qos=2048) == bad


def test_keep_refusals(L):
    for kw in (dict(keep=None), dict(keep=2), dict(n=None), dict(n=6), dict(lo=2), dict(ks=2), dict(ws=128, wsb=256)):
        assert keep(L, **kw) == qlin.ERR_INVALID_ARG, kw
    assert keep(L, s=step(T=33), ks=33) == qlin.ERR_UNSUPPORTED
    assert keep(L, ws=256, wsb=255) == qlin.ERR_WORKSPACE


def test_sample_refusals(L):
    def call(M=2, V=100, dtype=2, logits=4096, ld=100, u=4096, t=None, k=None, p=None, mp=None, token=4096, prob=None, flags=0):
        return L.qlin_sample(M, V, dtype, logits, ld, u, t, k, p, mp, token, prob, flags, None)

    bad = qlin.ERR_INVALID_ARG
    for kw in (dict(M=-1), dict(V=0), dict(dtype=1), dict(dtype=3), dict(logits=None), dict(logits=4098), dict(ld=99), dict(u=None),
               dict(u=2), dict(token=None), dict(token=2), dict(t=2), dict(k=2), dict(p=2), dict(mp=2), dict(prob=2), dict(flags=2)):
        assert call(**kw) == bad, kw
    assert call(V=524289, ld=524289) == qlin.ERR_UNSUPPORTED
    assert call(M=1 << 25) == qlin.ERR_UNSUPPORTED
    assert call(M=0, logits=None, u=None, token=None) == qlin.OK


@pytest.mark.parametrize("most", [8, 16])
def test_sample_plans_hold_every_row(L, most):
    """Whatever the number and the length of the rows, and whether the device holds clusters of 16 CTAs or of 8: no more
    CTAs than a cluster holds, and a slice that each has room for."""
    lengths = sorted({V + d for n in range(20) for V in (1 << n, 3 << n) for d in (-1, 0, 1)} | {32000, 131071, 262144, 300007, 524288})
    rows = sorted({1, 3, 5, 6, 7, 12, 20, 63, 65, 1000, 1 << 20, 1 << 24} | {1 << n for n in range(11)} | {9, 17, 19, 38, 76, 152})
    for V in (v for v in lengths if 1 <= v <= 524288):
        for M in rows:
            for dtype in (torch.float32, torch.bfloat16):
                for top_k in (False, True):
                    C, in_place = qlin.debug_sample_plan(M, V, dtype, top_k, most)
                    assert C in (1, 2, 4, 8, 16) and C <= most, (M, V, dtype, top_k)
                    assert C * (65536 if in_place else 32768) >= V, (M, V, dtype, top_k, C, in_place)
                    assert C > 1 or (not in_place and V <= 16384)
    for bad in ((0, 100, torch.float32, False, most), (1, 0, torch.float32, False, most), (1, 524289, torch.float32, False, most),
                (1, 100, torch.float16, False, most), (1, 100, torch.float32, False, 4)):
        with pytest.raises(qlin.QlinError):
            qlin.debug_sample_plan(*bad)


def test_sample_weight_export_refusals(L):
    one, z = torch.ones(1), torch.zeros(1)
    for x, m, t in ((2 * one, one, one), (math.nan * one, one, one), (z, math.inf * one, one), (z, one, z), (z, one, -one),
                    (z, one, math.nan * one)):
        with pytest.raises(qlin.QlinError):
            qlin.debug_sample_weight(x, m, t)
    assert L.qlin_debug_sample_weight(-1, None, None, None, None) == qlin.ERR_INVALID_ARG
    assert L.qlin_debug_sample_weight(1, None, None, None, None) == qlin.ERR_INVALID_ARG
    assert L.qlin_debug_sample_weight(0, None, None, None, None) == qlin.OK


def test_sample_weights_are_as_close_as_stated(L):
    """Weights above 2^-10 within 2.5 * 2^-31 of theirs, as the header says.  In units of 2^-31 of a weight 2^y, by the
    steps of its making: the table's entry 1/2, the product's cut-off part 1, z and the constant in it 1/32, the series'
    fp32 roundings (four of 2^-24 of z^2 / 2 < 2^-12) 1/8 and its first term left out (z^5 / 120) 1/11, y's two roundings
    (2^-32 together, times ln 2) 0.35, the last one to a multiple of 2^-42 (2^-43 / 2^-10) 1/4: 2.4.  Below: within half a
    unit of 2^-42 more."""
    g = torch.Generator().manual_seed(3)
    n = 400000
    T = torch.exp2(torch.rand(n, generator=g) * 40 - 20)
    mx = torch.randn(n, generator=g) * T * torch.exp2(torch.rand(n, generator=g) * 8 - 4)
    x = mx - T * torch.rand(n, generator=g) * 7.0
    x[::2] = mx[::2] - T[::2] * torch.rand(n // 2, generator=g) * 31.0
    have = qlin.debug_sample_weight(x, mx, T).numpy().astype(np.longdouble) / 2 ** 42
    a, b, t = (v.numpy().astype(np.longdouble) for v in (x, mx, T))
    want = np.exp((a - b) / t)
    off = np.abs(have - want)
    big = want >= 2.0 ** -10
    assert big.sum() > n // 3 and float((off[big] / want[big]).max()) <= 2.5 * 2.0 ** -31
    assert float((off - 2.5 * 2.0 ** -31 * want).max()) <= 2.0 ** -43
    # every entry of the table, every sign of what follows it
    y = -(np.arange(64)[:, None] + np.array([0.0, 1e-4, 0.25, 0.5, 0.75, 0.9999])) / 32
    x = torch.tensor(y * math.log(2), dtype=torch.float32)
    have = qlin.debug_sample_weight(x, torch.zeros(()), torch.ones(())).numpy().astype(np.longdouble) / 2 ** 42
    want = np.exp(x.numpy().astype(np.longdouble))
    assert float((np.abs(have - want) / want).max()) <= 2.5 * 2.0 ** -31


def test_sample_weights_of_differences_beyond_fp32(L):
    """Finite logits whose difference is above the largest fp32 have the weight that the temperature gives them; an
    infinite temperature gives all of them the same, a forbidden token none."""
    mx = torch.tensor([3e38, 3.4e38, 2e38, 3e38])
    x = torch.tensor([-3e38, -3.4e38, -1.9e38, -1e38])
    one = 1 << 42
    for T in (3.4e38, 1e38, 6e37, 3e37):
        T32 = float(torch.tensor(T))
        want = torch.exp((x.double() - mx.double()) / T32)
        have = qlin.debug_sample_weight(x, mx, torch.tensor(T32)).double() / one
        # 1 / T below 2^-126 is a multiple of 2^-149: half a unit of its 2^-128 and more, times y, two fp32 terms
        y = (want.log().abs() / math.log(2)).double()
        assert bool(((have - want).abs() <= want * (2.0 ** -21 * y * math.log(2) + 2.0 ** -29) + 1 / one).all()), (T, have, want)
    assert (qlin.debug_sample_weight(x, mx, torch.tensor(math.inf)) == one).all()
    assert (qlin.debug_sample_weight(torch.tensor(-math.inf), mx, torch.tensor([math.inf, 1.0, 1e38, 1e-40])) == 0).all()
    for T in (1e30, 1.0, 1e-40):  # too far below at these
        assert (qlin.debug_sample_weight(x, mx, torch.tensor(T)) == 0).all()


def test_rope_turns_are_exact_fractions(L):
    # whole, half and quarter turns per position; negative ones from the other side
    t = qlin.rope_turns(radians=[0.0, math.pi, math.pi / 2, -math.pi / 2, 2 * math.pi, 5 * math.pi], device="cpu")
    want = [0, 1 << 63, 1 << 62, 3 << 62, 0, 1 << 63]
    assert [int(x) & (2 ** 64 - 1) for x in t] == want
    t = qlin.rope_turns(1e6, 64, device="cpu")
    assert t.shape == (32,)
    for i, x in enumerate(t):
        assert int(x) / 2 ** 64 == pytest.approx(1e6 ** (-2 * i / 64) / (2 * math.pi), rel=2 ** -51)
    assert qlin.rope_turns(1e4, 0, device="cpu").shape == (0,)
    for kw in (dict(radians=[math.nan]), dict(radians=[math.inf]), dict(radians=[0.0] * 129)):
        with pytest.raises(qlin.QlinError):
            qlin.rope_turns(device="cpu", **kw)
    with pytest.raises(ValueError):
        qlin.rope_turns(1e4, 63)


def test_the_binding_refuses_what_it_can_see():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        qlin.KVCache(z(2, 4, 16, 64), z(2, 4, 16, 128))
    with pytest.raises(ValueError):
        qlin.KVCache(z(2, 4, 16, 64, dt=torch.float32), z(2, 4, 16, 64, dt=torch.float32))
    with pytest.raises(ValueError):
        qlin.KVCache(z(2, 4, 16, 64), z(2, 16, 4, 64).transpose(1, 2))
    with pytest.raises(ValueError):
        qlin.KVCache(z(2, 4, 64, 16).transpose(2, 3), z(2, 4, 64, 16).transpose(2, 3))
    c = qlin.KVCache(z(2, 4, 16, 64), z(2, 4, 16, 64))
    for kw in (dict(page_table=i32(3, 5)), dict(len=i32(2).long()), dict(count=i32(3)), dict(mask=i32(4)), dict(depth=i32(2, 4)),
               dict(mask=i32(3), depth=i32(2, 3)), dict(page_table=i32(5, 2).t())):
        with pytest.raises(ValueError):
            qlin.KVStep(**{**dict(page_table=i32(2, 5), len=i32(2), T=3), **kw})
    s = qlin.KVStep(i32(2, 5), i32(2), 3)
    for call in (lambda: qlin.tree_attention(c, s, z(6, 512)), lambda: qlin.kv_append(c, s, q=z(6, 512)),
                 lambda: qlin.kv_keep(c, s, i32(2, 3), i32(2)), lambda: qlin.sample(z(2, 9), z(2, dt=torch.float32))):
        with pytest.raises(ValueError, match="not on a GPU"):  # there is no CPU path
            call()


def test_the_package_imports_on_a_torch_without_cuda():
    """Such a torch has no raw device and stream getters; calls on tensors are refused as on any machine without a GPU."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from w6a8_quantized_linear_gb300 import qlin
try:
    qlin.sample(torch.zeros(2, 9), torch.zeros(2))
except ValueError as e:
    assert "not on a GPU" in str(e)
else:
    raise SystemExit("not refused")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
