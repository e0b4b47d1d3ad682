"""Penalties, biases and grammar masks on logits on the GPU against a plain 64-bit form."""
import math

import numpy as np
import pytest
import torch

from gpu_util import DEV, built
from test_gpu_step import i32
from w6a8_quantized_linear_gb300 import qlin

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built()
    torch.cuda.set_device(DEV)


def reference(x, history, prompt, path, r, p, f, biases, allowed):
    """One row in 64 bits, and the sum of the magnitudes that the kernel rounds on the way (each once, to fp32)."""
    V = len(x)
    y, size = x.astype(np.float64), np.zeros(V)
    seen, made = np.zeros(V, bool), np.zeros(V, np.int64)
    for i, v in enumerate(list(history) + list(path)):
        if 0 <= v < V:
            seen[v] = True
            made[v] += i >= prompt
    if not r > 0:
        r = 1.0
    with np.errstate(invalid="ignore"):
        y[seen] = np.where(y[seen] > 0, y[seen] / r, y[seen] * r)
        size[seen] += abs(y[seen])
        n = made > 0
        size[n] += f * made[n] + abs(y[n] - f * made[n]) + abs(y[n] - f * made[n] - p)
        y[n] = y[n] - f * made[n] - p
        total = {}
        for v, b in biases:
            if 0 <= v < V:
                total.setdefault(v, []).append(b)
        for v, bs in total.items():  # of one token: added up first
            size[v] += sum(abs(sum(bs[:i + 1])) for i in range(1, len(bs))) + abs(y[v] + sum(bs))
            y[v] += sum(bs)
    size = np.where(np.isfinite(size), size, 0)
    if allowed is not None:
        bits = (allowed[np.arange(V) // 32].astype(np.int64) >> (np.arange(V) % 32)) & 1
        y[bits == 0] = -np.inf
    return y, size


class Case:
    def __init__(self, B, T, V, L, dtype, seed=0, n_bias=0, allowed=None, drafts=False, pad=0, twice=False, spread=5.0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.V, self.L = B, T, V, L
        self.wide = torch.full((B * T, V + pad), math.nan)
        self.wide[:, :V] = torch.randn(B * T, V, generator=g) * 3
        self.wide = self.wide.to(dtype)
        self.logits = self.wide[:, :V]
        tokens = lambda *s: (torch.rand(*s, generator=g) ** spread * V).int()  # noqa: E731
        self.history = torch.where(torch.rand(B, L, generator=g) < 0.02, V + 3, tokens(B, L)).int()
        self.history[torch.rand(B, L, generator=g) < 0.02] = -1
        self.n = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
        self.n[0] = L
        self.prompt = (self.n.float() * torch.rand(B, generator=g)).int()
        self.r, self.p, self.f = 0.7 + torch.rand(B, generator=g), torch.rand(B, generator=g), torch.rand(B, generator=g) * 0.3
        self.draft = self.mask = None
        if drafts:
            self.draft = tokens(B, T)
            if T > 2:
                self.draft[:, 2] = self.draft[:, 0]  # a token twice on a path
            self.mask = torch.tensor([(1 << t) | (torch.randint(0, 1 << 30, (1,), generator=g).item() & ((1 << t) - 1)) for t in range(T)])
            self.mask = torch.where(self.mask >= 1 << 31, self.mask - (1 << 32), self.mask).int()
        self.bt = self.bv = None
        if n_bias:
            self.bt = torch.randint(-2, V + 2, (B, n_bias), generator=g, dtype=torch.int32)
            if twice:
                self.bt[:, 1::2] = self.bt[:, 0::2][:, : self.bt[:, 1::2].shape[1]]
                self.bt[:, -1] = self.bt[:, 0]
            self.bv = torch.randn(B, n_bias, generator=g) * 5
        self.allowed = None
        if allowed is not None:
            words = torch.rand(B * T, -(-V // 32), 32, generator=g) < allowed
            words = (words.long() << torch.arange(32)).sum(-1)
            self.allowed = torch.where(words >= 1 << 31, words - (1 << 32), words).int()

    def args(self, dev=DEV):
        a = dict(history=self.history, history_len=self.n, prompt_len=self.prompt, draft=self.draft, mask=self.mask,
                 repetition=self.r, presence=self.p, frequency=self.f, bias_token=self.bt, bias=self.bv, allowed=self.allowed)
        return {k: None if v is None else v.to(dev) for k, v in a.items()}

    def check(self, got, rows=None):
        got = got.cpu().double().numpy()
        for m in rows if rows is not None else range(self.B * self.T):
            b, t = divmod(m, self.T)
            path = []
            if self.draft is not None:
                path = [int(self.draft[b, j]) for j in range(self.T) if int(self.mask[t]) >> j & 1]
            biases = [] if self.bt is None else list(zip(self.bt[b].tolist(), self.bv[b].double().tolist()))
            want, size = reference(self.logits[m].double().numpy(), self.history[b, : int(self.n[b])].tolist(), int(self.prompt[b]),
                                   path, float(self.r[b]), float(self.p[b]), float(self.f[b]), biases,
                                   None if self.allowed is None else self.allowed[m].numpy())
            banned = want == -np.inf
            assert np.array_equal(got[m] == -np.inf, banned)
            with np.errstate(invalid="ignore"):
                off = np.abs(got[m] - want)[~banned]
            bound = 1.001 * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(want) if self.logits.dtype == BF else 0)
            assert (off <= bound[~banned] + 1e-38).all(), (m, (off - bound[~banned]).max())
            same = ~banned & (size == 0)
            assert np.array_equal(got[m][same], self.logits[m].double().numpy()[same])


CASES = [
    # B, T, V, L, dtype, n_bias, allowed, drafts, pad, twice
    (1, 1, 32000, 311, F32, 0, None, False, 0, False),
    (1, 1, 1, 1, F32, 1, None, False, 0, False),
    (2, 1, 33, 7, BF, 3, 0.5, False, 3, True),
    (1, 8, 131071, 20011, F32, 64, 0.33, True, 0, False),
    (3, 5, 1001, 5000, BF, 300, 0.9, True, 0, True),
    (2, 32, 4099, 4097, F32, 1024, None, True, 5, True),
    (5, 3, 50257, 9000, BF, 20, 0.001, True, 7, False),
    (1, 1, 524288, 60000, BF, 0, 0.5, False, 0, False),
    (7, 1, 70001, 1, F32, 0, 0.0, False, 1, False),
    (2, 70, 999, 50, F32, 4, 0.5, False, 1, False),
    (70, 1, 20000, 9999, BF, 3, None, True, 0, False),
]


@pytest.mark.parametrize("place", ["new", "in place", "unaligned"])
@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_adjust_against_64_bits(case, place):
    B, T, V, L, dtype, n_bias, allowed, drafts, pad, twice = case
    c = Case(B, T, V, L, dtype, n_bias + V, n_bias, allowed, drafts, pad, twice)
    wide = c.wide.to(DEV)
    logits, before = wide[:, :V], c.wide.clone()
    out = None
    if place == "in place":
        out = logits
    elif place == "unaligned":  # rows of another stride and alignment than the logits'
        out = torch.full((B * T, V + 9), 7.0, dtype=dtype, device=DEV)[:, 3:3 + V]
    got = qlin.adjust_logits(logits, out=out, **c.args())
    c.check(got)
    if place != "in place":
        assert torch.equal(wide.cpu().nan_to_num(nan=9.0), before.nan_to_num(nan=9.0))
    elif pad:
        assert wide[:, V:].isnan().all()


def test_parts_alone():
    """Each operand on its own; none at all is a copy."""
    c = Case(2, 3, 777, 40, F32, 3, 9, 0.5, True)
    x, a = c.logits.to(DEV), c.args()
    assert torch.equal(qlin.adjust_logits(x), x)
    nothing = torch.zeros(0)
    for keep in (("history", "history_len", "prompt_len", "repetition"), ("history", "frequency"), ("draft", "mask", "presence"),
                 ("bias_token", "bias"), ("allowed",), ("history", "draft", "mask"), ("history_len", "presence")):
        d = Case(2, 3, 777, 40, F32, 3, 9, 0.5, True)
        d.n = d.n if "history_len" in keep else torch.full((2,), 40)
        d.prompt = d.prompt if "prompt_len" in keep else torch.zeros(2, dtype=torch.int32)
        if "history" not in keep:
            d.history = d.history[:, :0]
        d.draft = d.draft if "draft" in keep else None
        d.r = d.r if "repetition" in keep else torch.ones(2)
        d.p = d.p if "presence" in keep else torch.zeros(2)
        d.f = d.f if "frequency" in keep else torch.zeros(2)
        d.bt = d.bt if "bias" in keep else None
        d.allowed = d.allowed if "allowed" in keep else None
        d.check(qlin.adjust_logits(x, **{k: a[k] for k in keep}))
    assert nothing.numel() == 0


def test_values_that_are_not_ordinary():
    """Infinite and NaN logits, penalties that are none, and what the rules leave alone."""
    inf, nan = math.inf, math.nan
    x = torch.tensor([[inf, -inf, nan, 1.0, -1.0, 0.0, inf, -inf, nan, 5.0]] * 3, device=DEV)
    history = i32([[0, 1, 2, 3, 4, 5]] * 3)
    r = torch.tensor([2.0, nan, -1.0], device=DEV)
    got = qlin.adjust_logits(x, history=history, prompt_len=i32([6, 6, 6]), repetition=r).cpu()
    want = torch.tensor([[inf, -inf, nan, 0.5, -2.0, 0.0, inf, -inf, nan, 5.0]] + [x[0].tolist()] * 2)
    assert torch.equal(got.nan_to_num(nan=9.0), want.nan_to_num(nan=9.0)) and torch.equal(got.isnan(), want.isnan())
    # a forbidden NaN is forbidden, an allowed one stays; no mask bit touches its neighbours
    allowed = i32([[0b0111111011]])
    got = qlin.adjust_logits(x[:1], allowed=allowed).cpu()[0]
    assert got[2] == -inf and got[9] == -inf and got[8].isnan() and got[0] == inf and got[3] == 1.0
    # one list of biases and one mask for all rows
    got = qlin.adjust_logits(x, bias_token=i32([3, 3, 9]), bias=torch.tensor([1.0, 2.0, -5.0], device=DEV), allowed=i32([1 << 3 | 1 << 9]))
    assert torch.equal(got.cpu()[:, 3], torch.full((3,), 4.0)) and torch.equal(got.cpu()[:, 9], torch.zeros(3))
    assert (got.cpu()[:, [0, 1, 2, 4, 5, 6, 7, 8]] == -inf).all()


def test_a_history_of_one_token_many_times():
    """The longest history, all of it one token: a count of a million."""
    L, V = 1000000, 40000
    h = torch.full((2, L), 17, dtype=torch.int32, device=DEV)
    h[1, : L // 2] = V - 1
    x = torch.zeros(2, V, device=DEV)
    got = qlin.adjust_logits(x, history=h, frequency=torch.tensor([1.0, 1.0], device=DEV), prompt_len=i32([0, 3]))
    want = torch.zeros(2, V)
    want[0, 17], want[1, 17], want[1, V - 1] = -L, -(L // 2), -(L // 2 - 3)
    assert torch.equal(got.cpu(), want)


def test_replay_streams_and_then_sampling():
    """Captured with the sampler behind it: histories, lengths and masks are read at replay; another stream."""
    c = Case(4, 1, 30000, 6000, F32, 8, 16, 0.2)
    a = c.args()
    x, out, u = c.logits.to(DEV), torch.empty(4, 30000, device=DEV), torch.full((4,), 0.5, device=DEV)
    token = torch.empty(4, dtype=torch.int32, device=DEV)
    cold = torch.zeros(4, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            qlin.adjust_logits(x, out=out, flags=qlin.FLAG_PDL, **a)
            qlin.sample(out, u, temperature=cold, token=token, flags=qlin.FLAG_PDL)
    for seed in (21, 22):
        d = Case(4, 1, 30000, 6000, F32, seed, 16, 0.2)
        x.copy_(d.logits)
        for k, v in d.args().items():
            if v is not None:
                a[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        d.check(out)
        assert torch.equal(token.long(), out.argmax(1))
    other = torch.empty_like(out)
    with torch.cuda.stream(side):
        qlin.adjust_logits(x, out=other, **a)
    side.synchronize()
    assert torch.equal(other, out)


def test_lengths_and_tokens_far_outside():
    """Lengths below 0 and above the history's width, tokens at the ends of their type, prompts of any length."""
    V = 5000
    h = i32([[-2 ** 31, 2 ** 31 - 1, 7, V, -1, 4999, 7, 0]] * 4)
    x = torch.zeros(4, V, device=DEV)
    one = torch.ones(4, device=DEV)
    got = qlin.adjust_logits(x, history=h, history_len=i32([8, 2 ** 31 - 1, -2 ** 31, 3]), prompt_len=i32([-2 ** 31, 6, 0, 2 ** 31 - 1]),
                             frequency=one).cpu()
    want = torch.zeros(4, V)
    want[0, 7], want[0, 4999], want[0, 0] = -2, -1, -1
    want[1, 7], want[1, 0] = -1, -1
    assert torch.equal(got, want)
    long = h.repeat(1, 700)  # the same, by clusters
    got = qlin.adjust_logits(x, history=long, history_len=i32([8, 2 ** 31 - 1, -2 ** 31, 3]),
                             prompt_len=i32([-2 ** 31, 5598, 0, 2 ** 31 - 1]), frequency=one).cpu()
    assert torch.equal(got, want)


def test_more_rows_than_sequences():
    """Rows that nothing tells apart, more of them than a call has sequences, from the logits' own memory and from a slice."""
    M, V = 66000, 100
    wide = torch.randn(M, V + 4, generator=torch.Generator().manual_seed(3)).bfloat16()
    allowed = torch.randint(-2 ** 31, 2 ** 31, (M, 4), generator=torch.Generator().manual_seed(4), dtype=torch.int64).int()
    bits = (allowed.long()[:, torch.arange(V) // 32] >> torch.arange(V) % 32) & 1
    for x in (wide.to(DEV)[:, :V], wide[:, :V].contiguous().to(DEV)):
        want = torch.where(bits == 1, wide[:, :V].float(), -math.inf)
        want[:, 7] += torch.where(bits[:, 7] == 1, 2.0, 0.0)
        for out in (None, torch.empty(M, V, dtype=BF, device=DEV)):
            got = qlin.adjust_logits(x, out=out, allowed=allowed.to(DEV), bias_token=i32([7]), bias=torch.tensor([2.0], device=DEV))
            assert torch.equal(got.cpu(), want.bfloat16())


def test_arguments_of_the_two_ways_agree():
    """The same operands as plain tensors (read by the extension) and as slices of wider ones (read one by one)."""
    c = Case(3, 4, 5003, 600, F32, 11, 40, 0.5, True)
    a = c.args()
    x = c.logits.to(DEV)
    plain = qlin.adjust_logits(x, out=torch.empty_like(x), **a)
    slices = {}
    for k, t in a.items():
        if t is None or t.dim() < 2 or k in ("draft", "mask"):
            slices[k] = t
            continue
        wide = torch.zeros(t.shape[0], t.shape[1] + 3, dtype=t.dtype, device=DEV)
        wide[:, 2:-1] = t
        slices[k] = wide[:, 2:-1]
    assert torch.equal(qlin.adjust_logits(x, **slices), plain)
    with pytest.raises(ValueError):
        qlin.adjust_logits(x, out=torch.empty_like(x), **{**a, "history": a["history"].long()})
    with pytest.raises(ValueError):
        qlin.adjust_logits(x, out=torch.empty_like(x), **{**a, "presence": a["presence"][:2]})
    with pytest.raises(ValueError, match="cpu"):
        qlin.adjust_logits(x, out=torch.empty_like(x), **{**a, "allowed": a["allowed"].cpu()})
    with pytest.raises(qlin.QlinError):
        qlin.adjust_logits(x.half(), out=torch.empty_like(x.half()), **a)
    c.check(plain)


@pytest.mark.parametrize("n", [3, 40, 700])
def test_biases_of_one_token_are_added_to_one_another_first(n):
    """In the list's order, in fp32: of 1e8, 1 and -1e8 nothing is left to be added to the logit."""
    V = 5000
    x = torch.ones(2, V, device=DEV)
    token, bias = torch.arange(100, 100 + n, dtype=torch.int32).repeat(2, 1), torch.zeros(2, n)
    token[:, [0, n // 2, n - 1]] = i32([7, 7, 7]).cpu()
    bias[0, [0, n // 2, n - 1]] = torch.tensor([1e8, 1.0, -1e8])
    bias[1, [0, n // 2, n - 1]] = torch.tensor([1e8, -1e8, 1.0])
    got = qlin.adjust_logits(x, bias_token=token.to(DEV), bias=bias.to(DEV)).cpu()
    want = torch.ones(2, V)
    want[1, 7] = 2.0
    assert torch.equal(got, want)


def test_operands_of_no_width():
    """A history or lists of biases of width 0: as if not given; through both ways of the binding."""
    x = torch.randn(6, 500, generator=torch.Generator().manual_seed(1)).to(DEV)
    none, nothing = torch.zeros(2, 0, dtype=torch.int32, device=DEV), torch.zeros(2, 0, device=DEV)
    one = torch.ones(2, device=DEV)
    for kw in (dict(history=none, presence=one, repetition=2 * one), dict(history=none, history_len=i32([0, 5]), prompt_len=i32([3, 0]), frequency=one),
               dict(bias_token=none, bias=nothing), dict(bias_token=none[0], bias=nothing[0]), dict(history=none, bias_token=none, bias=nothing)):
        assert torch.equal(qlin.adjust_logits(x, **kw), x)
        assert torch.equal(qlin.adjust_logits(x, out=torch.empty_like(x), **kw), x)
        y = x.clone()
        assert qlin.adjust_logits(y, out=y, **kw) is y and torch.equal(y, x)
        draft = i32([[3, 4, 3], [9, 9, 9]])  # beside them, what does count
        got = qlin.adjust_logits(x, **kw, draft=draft, **({} if "presence" in kw else dict(presence=one)))
        want = x.clone()
        for m in range(6):
            for v in set(draft[m // 3, : m % 3 + 1].tolist()):
                y = want[m, v]
                if "repetition" in kw:
                    y = y / 2 if y > 0 else y * 2
                n = draft[m // 3, : m % 3 + 1].tolist().count(v)
                want[m, v] = y - (n if "frequency" in kw else 0) - 1
        assert torch.equal(got, want)


@pytest.mark.parametrize("case", [(2, 3, 20000, 6000, F32, 9, 0.7), (3, 40, 9001, 5000, BF, 0, None), (40, 2, 33001, 33000, BF, 3, None),
                                  (40, 2, 131071, 8000, F32, 3, None)], ids=["0", "1", "2", "3"])
def test_several_rows_without_drafts_under_a_long_history(case):
    """By clusters, where these make one round of blocks or the history is very long; by single blocks else."""
    B, T, V, L, dtype, n_bias, allowed = case
    c = Case(B, T, V, L, dtype, V, n_bias, allowed)
    x = c.logits.to(DEV)
    got = qlin.adjust_logits(x, **c.args())
    c.check(got, rows=sorted({0, 1, B * T - 1, B * T // 2}))
    qlin.adjust_logits(x, out=x, **c.args())
    assert torch.equal(x, got)


@pytest.mark.parametrize("case", [(2, 1, 50000, F32, False), (64, 1, 131071, BF, False), (3, 5, 20000, BF, True), (1, 8, 131071, F32, True)],
                         ids=["0", "1", "2", "3"])
def test_a_history_much_wider_than_its_lengths(case):
    """The same values as from a history cut to them; what lies behind the lengths is anything."""
    B, T, V, dtype, drafts = case
    c = Case(B, T, V, 1000, dtype, 5, 4, None, drafts)
    a = c.args()
    x = c.logits.to(DEV)
    want = qlin.adjust_logits(x, **a)
    c.check(want, rows=sorted({0, B * T - 1}))
    wide = torch.randint(0, V, (B, 40000), generator=torch.Generator().manual_seed(6), dtype=torch.int32)
    wide[:, :1000] = c.history
    assert torch.equal(qlin.adjust_logits(x, **{**a, "history": wide.to(DEV)}), want)
