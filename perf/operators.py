"""The operators of a decode / tree-verification step around the quantised linears: what is measured of them.

Four operators: ``kv_append`` (per-head norms and position rotation of the projected q and k, k and v stored into a
paged cache), ``tree_attention`` (a tree of drafted tokens, or one token, over that cache), ``kv_keep`` (the accepted
path of a verified tree moves up behind the committed tokens) and ``sample`` (temperature, top-k, top-p, min-p from
given uniform numbers).  ``run`` computes them in plain torch operations, or, where ``own`` is true, by the
framework's calls; ``exact`` in 64 bits.
"""
import math

import numpy as np
import torch

own = False

THETA = 1.0e6   # base of the rotation's frequencies
EPS = 1.0e-6    # of the norms
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # the projections of one decoded token: the smallest append, bound by its launch
        dict(name="append_token", op="append", B=1, T=1, Hq=24, Hkv=4, D=256, rot=64, pairs=False, src="f32", cache="bf16",
             page=64, len=2000),
        # a tree of eight rows, the widest step of the linears
        dict(name="append_tree", op="append", B=1, T=8, Hq=48, Hkv=8, D=128, rot=128, pairs=False, src="f32", cache="bf16",
             page=16, len=40961),
        # a prompt's rows behind a shared prefix, an odd number of them
        dict(name="append_prompt", op="append", B=1, T=4001, Hq=48, Hkv=8, D=128, rot=128, pairs=True, src="f32",
             cache="f16", page=32, len=517),
        # one token over a short chat
        dict(name="attention_token", op="attention", B=1, T=1, Hq=24, Hkv=4, D=256, cache="bf16", page=64, len=1777),
        # an eight-row tree over an ordinary context, ending inside a page
        dict(name="attention_tree", op="attention", B=1, T=8, Hq=48, Hkv=8, D=128, cache="bf16", page=16, len=8190),
        # an eight-row tree over a book: the largest cache
        dict(name="attention_tree_long", op="attention", B=1, T=8, Hq=24, Hkv=4, D=256, cache="bf16", page=64, len=130999),
        # several requests of different lengths, three rows each
        dict(name="attention_batch", op="attention", B=8, T=3, Hq=48, Hkv=8, D=128, cache="f16", page=32, len=30011),
        # the accepted branch of one tree
        dict(name="keep_one", op="keep", B=1, T=8, Hkv=8, D=128, cache="bf16", page=16, len=8190),
        # the accepted branches of a batch of larger trees
        dict(name="keep_batch", op="keep", B=24, T=16, Hkv=8, D=128, cache="bf16", page=32, len=2011),
        # one token from a small vocabulary
        dict(name="sample_token", op="sample", M=1, V=32000, dtype="f32", top_k=False, top_p=True, min_p=False, banned=0.0),
        # every row of a tree, all filters, an odd vocabulary, some tokens forbidden
        dict(name="sample_tree", op="sample", M=8, V=131071, dtype="f32", top_k=True, top_p=True, min_p=True, banned=0.1),
        # a large batch of 16-bit logits (many equal ones) over a large vocabulary
        dict(name="sample_batch", op="sample", M=64, V=262144, dtype="bf16", top_k=True, top_p=True, min_p=False, banned=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "keep", "sample", "sample"])
    if op == "sample":
        return dict(op=op, M=_log_int(rng, 1, 64), V=_log_int(rng, 500, 262144), dtype=rng.choice(["f32", "bf16"]),
                    top_k=rng.random() < 0.6, top_p=rng.random() < 0.6, min_p=rng.random() < 0.4,
                    banned=rng.choice([0.0, 0.1, 0.5]))
    D, Hkv = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 5, 8])
    case = dict(op=op, B=1, T=1, Hkv=Hkv, D=D, cache=rng.choice(["bf16", "f16"]), page=rng.choice([16, 32, 64, 128]), len=0)
    if op == "append":
        case["Hq"] = Hkv * rng.choice([1, 2, 3, 6, 8])
        case["rot"] = rng.choice([D, D // 2, D // 4])
        case["pairs"] = rng.random() < 0.5
        case["src"] = rng.choice(["f32", "bf16"])
        case["T"] = _log_int(rng, 1, 2000)
        case["B"] = rng.choice([1, 1, 2, 3]) if case["T"] > 32 else rng.choice([1, 1, 2, 8, 13])
        case["len"] = _log_int(rng, 1, 60000 // case["B"])
    elif op == "attention":
        g = rng.choice([1, 2, 3, 6, 8])
        case["Hq"] = Hkv * g
        case["T"] = rng.choice([1, 1, 2, 3, 5, 8, 8, 16])
        case["B"] = rng.choice([1, 1, 1, 2, 5, 8, 19])
        case["len"] = _log_int(rng, 1, 131000 * 1024 // (Hkv * D) // case["B"] // (1 + case["T"] // 16))
        case["len"] = max(1, min(case["len"], 200000))
    else:
        case["T"] = rng.choice([2, 4, 5, 8, 8, 16, 32])
        case["B"] = rng.choice([1, 1, 3, 8, 31])
        case["len"] = _log_int(rng, 1, 8000)
    return case


def _lens(case):
    """The sequences' committed tokens: the first the longest, down to a quarter of it."""
    B, n = case["B"], case["len"]
    return [max(1, n - (3 * n * b) // (4 * B)) for b in range(B)]


def _tree(T):
    """Parents of a drafted tree's rows: row 0 the committed token, then two branches, each a chain."""
    half = 1 + (T - 1 + 1) // 2
    return [-1] + [0 if t in (1, half) else t - 1 for t in range(1, T)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"op": case["op"], "case": case}
    if case["op"] == "sample":
        M, V = case["M"], case["V"]
        logits = torch.randn(M, V, device=dev, generator=g) * 2.5
        lift = torch.randint(0, V, (M, 12), device=dev, generator=g)  # the few likely continuations
        logits.scatter_(1, lift, 6 + 5 * torch.rand(M, 12, device=dev, generator=g))
        if case["banned"]:
            logits.masked_fill_(torch.rand(M, V, device=dev, generator=g) < case["banned"], -math.inf)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["u"] = torch.rand(M, device=dev, generator=g)
        s["temperature"] = 0.6 + 0.7 * torch.rand(M, device=dev, generator=g)
        if M > 3:
            s["temperature"][M // 2] = 0  # a request that decodes greedily
        s["top_k"] = torch.randint(1, min(V, 400), (M,), device=dev, generator=g, dtype=torch.int32) if case["top_k"] else None
        s["top_p"] = 0.7 + 0.29 * torch.rand(M, device=dev, generator=g) if case["top_p"] else None
        s["min_p"] = 0.01 + 0.1 * torch.rand(M, device=dev, generator=g) if case["min_p"] else None
        s["token"] = torch.empty(M, dtype=torch.int32, device=dev)
        s["prob"] = torch.empty(M, dtype=torch.float32, device=dev)
        return s
    B, T, Hkv, D, page = case["B"], case["T"], case["Hkv"], case["D"], case["page"]
    dt = DTYPES[case["cache"]]
    per = -(-(case["len"] + T) // page)
    pages = B * per + 3
    s["k"] = torch.randn(pages, Hkv, page, D, device=dev, generator=g, dtype=dt)
    s["v"] = torch.randn(pages, Hkv, page, D, device=dev, generator=g, dtype=dt)
    s["table"] = torch.randperm(pages, device=dev, generator=g)[: B * per].view(B, per).to(torch.int32)
    s["len"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
    if T <= 32:
        parent = _tree(T)
        depth, mask = [0], [1]
        for t in range(1, T):
            depth.append(depth[parent[t]] + 1)
            mask.append(mask[parent[t]] | 1 << t)
        s["depth"] = torch.tensor(depth, dtype=torch.int32, device=dev)
        s["mask"] = torch.tensor([m - (1 << 32) if m >> 31 else m for m in mask], dtype=torch.int32, device=dev)
    else:  # a prompt's rows follow one another
        s["depth"] = s["mask"] = None
    if case["op"] == "append":
        src, Hq = DTYPES[case["src"]], case["Hq"]
        s["q_in"] = torch.randn(B * T, Hq * D, device=dev, generator=g).mul_(1.7).to(src)
        s["k_in"] = torch.randn(B * T, Hkv * D, device=dev, generator=g).mul_(2.3).to(src)
        s["v_in"] = torch.randn(B * T, Hkv * D, device=dev, generator=g).to(src)
        s["q_gamma"] = 0.5 + torch.rand(D, device=dev, generator=g)
        s["k_gamma"] = 0.5 + torch.rand(D, device=dev, generator=g)
        s["q"] = torch.empty(B * T, Hq * D, dtype=dt, device=dev)
    elif case["op"] == "attention":
        s["q"] = torch.randn(B * T, case["Hq"] * D, device=dev, generator=g).to(dt)
        s["out"] = torch.empty(B * T, case["Hq"] * D, dtype=torch.bfloat16, device=dev)
    else:
        # the second branch is accepted, up to a length of its own for each sequence: its rows lie behind the places
        # that they move to
        n = 1 + (T - 1) // 2
        second = 1 + T // 2
        path = [0] + [second + i for i in range(n - 1)]
        s["keep"] = torch.tensor([path + [0] * (T - n)] * B, dtype=torch.int32, device=dev)
        s["n_keep"] = torch.randint(1, n + 1, (B,), device=dev, generator=g, dtype=torch.int32)
        s["len_out"] = torch.empty(B, dtype=torch.int32, device=dev)
    if own:
        from w6a8_quantized_linear_gb300 import qlin
        s["cache"] = qlin.KVCache(s["k"], s["v"])
        s["step"] = qlin.KVStep(s["table"], s["len"], T, depth=s["depth"], mask=s["mask"])
        if case["op"] == "append":
            s["turns"] = qlin.rope_turns(THETA, case["rot"], device=dev)
        if case["op"] == "attention":
            s["ws"] = qlin.new_workspace(qlin.tree_attention_workspace_bytes(s["cache"], B, T, case["Hq"]), dev)
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------------

def _rotate(x, pos, rot, pairs):
    """Rotate the first ``rot`` elements of x [rows, H, D] (fp32) by pos [rows]; the angles in 64 bits."""
    freq = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=x.device) / rot)
    angle = pos.double()[:, None] * freq
    c, n = angle.cos().float()[:, None], angle.sin().float()[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    if pairs:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2), rest], -1)
    a, b = head[..., : rot // 2], head[..., rot // 2:]
    return torch.cat([a * c - b * n, b * c + a * n, rest], -1)


def _places(s, at):
    """Page and row in the page of the tokens at [B, n]."""
    page = s["case"]["page"]
    return s["table"].long().gather(1, at // page), at % page


def _plain_append(s):
    c = s["case"]
    B, T, D, dt = c["B"], c["T"], c["D"], DTYPES[c["cache"]]
    ahead = torch.arange(T, device=s["len"].device)
    depth = ahead if s["depth"] is None else s["depth"].long()
    pos = (s["len"].long()[:, None] + depth).flatten()

    def normed(x, gamma):
        x = x.view(B * T, -1, D).float()
        return x * gamma / (x.square().mean(-1, keepdim=True) + EPS).sqrt()

    q = _rotate(normed(s["q_in"], s["q_gamma"]), pos, c["rot"], c["pairs"])
    k = _rotate(normed(s["k_in"], s["k_gamma"]), pos, c["rot"], c["pairs"])
    p, r = _places(s, s["len"].long()[:, None] + ahead)
    s["k"][p.flatten(), :, r.flatten()] = k.to(dt)
    s["v"][p.flatten(), :, r.flatten()] = s["v_in"].view(B * T, -1, D).to(dt)
    return {"q": q.reshape(B * T, -1).to(dt), "k": s["k"], "v": s["v"]}


def _plain_attention(s):
    c = s["case"]
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    g = Hq // Hkv

    def gathered(x):  # [B, Hkv, tokens, D]
        return x[s["table"].long()].transpose(1, 2).reshape(B, Hkv, -1, D).float()

    q = s["q"].view(B, T, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * T, D).float()
    k = gathered(s["k"])
    score = (q @ k.transpose(-1, -2)) * D ** -0.5
    score = score.view(B, Hkv, g, T, -1)
    draft = torch.arange(k.shape[2], device=k.device) - s["len"].long()[:, None]  # [B, tokens]
    bit = s["mask"].long()[:, None, None] >> draft.clamp(0, 31) & 1              # [T, B, tokens]
    seen = (draft < 0) | ((draft < T) & (bit == 1))
    score = torch.where(seen.transpose(0, 1)[:, None, None], score, -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    o = w.view(B, Hkv, g * T, -1) @ gathered(s["v"])
    return o.view(B, Hkv, g, T, D).permute(0, 3, 1, 2, 4).reshape(B * T, Hq * D).to(torch.bfloat16)


def _plain_keep(s):
    T = s["case"]["T"]
    i = torch.arange(T, device=s["len"].device)
    kept = i < s["n_keep"][:, None]
    base = s["len"].long()[:, None]
    src = torch.where(kept, s["keep"].long(), i)  # the others stay where they are
    sp, sr = _places(s, base + src)
    dp, dr = _places(s, base + i)
    for x in (s["k"], s["v"]):
        x[dp, :, dr] = x[sp, :, sr]
    return {"k": s["k"], "v": s["v"], "len": (s["len"] + s["n_keep"]).to(torch.int32)}


def _plain_sample(s):
    x = s["logits"].float()
    M, V = x.shape
    top = x.amax(1, keepdim=True)
    greedy = s["temperature"][:, None] <= 0
    t = torch.where(greedy, 1.0, s["temperature"][:, None]).double()
    w = torch.exp((x.double() - top.double()) / t)
    w = torch.where(greedy, (x == top).double(), w)
    _, order = torch.sort(x, dim=1, descending=True, stable=True)
    ranked = w.gather(1, order)
    rank = torch.arange(V, device=x.device)
    kept = torch.ones(M, V, dtype=torch.bool, device=x.device)
    if s["top_k"] is not None:
        kept &= rank < s["top_k"].long()[:, None]
    if s["top_p"] is not None:
        mass = torch.where(kept, ranked, 0.0)
        before = mass.cumsum(1) - mass
        kept &= before < s["top_p"].double()[:, None] * mass.sum(1, keepdim=True)
    if s["min_p"] is not None:
        kept &= ranked >= s["min_p"].double()[:, None]
    kept &= ~greedy | (rank == 0)
    kept = torch.zeros_like(kept).scatter_(1, order, kept)  # in the vocabulary's order
    mass = torch.where(kept, w, 0.0)
    total = mass.sum(1, keepdim=True)
    past = (mass.cumsum(1) > s["u"].double()[:, None] * total) & (mass > 0)
    last = torch.where(mass > 0, rank, -1).amax(1)
    token = torch.where(past.any(1), past.int().argmax(1), last)
    return {"token": token.to(torch.int32), "prob": (mass.gather(1, token[:, None]) / total).squeeze(1).float()}


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "keep": _plain_keep, "sample": _plain_sample}[s["op"]](s)
    from w6a8_quantized_linear_gb300 import qlin
    if s["op"] == "append":
        c = s["case"]
        qlin.kv_append(s["cache"], s["step"], q=s["q_in"], k=s["k_in"], v=s["v_in"], q_gamma=s["q_gamma"], k_gamma=s["k_gamma"],
                       eps=EPS, turns=s["turns"], pairs=c["pairs"], q_out=s["q"])
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    if s["op"] == "attention":
        return qlin.tree_attention(s["cache"], s["step"], s["q"], out=s["out"], ws=s["ws"])
    if s["op"] == "keep":
        qlin.kv_keep(s["cache"], s["step"], s["keep"], s["n_keep"], len_out=s["len_out"])
        return {"k": s["k"], "v": s["v"], "len": s["len_out"]}
    qlin.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                token=s["token"], prob=s["prob"])
    return {"token": s["token"], "prob": s["prob"]}


def work(case):
    if case["op"] == "sample":
        n = case["M"] * case["V"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2), "flops": 4 * n}
    B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
    if case["op"] == "append":
        values = B * T * (case["Hq"] + 2 * Hkv) * D
        return {"bytes": values * ((4 if case["src"] == "f32" else 2) + 2), "flops": 8 * B * T * (case["Hq"] + Hkv) * D}
    if case["op"] == "attention":
        tokens = sum(_lens(case)) + B * T
        return {"bytes": 2 * 2 * tokens * Hkv * D + 2 * 2 * B * T * case["Hq"] * D, "flops": 4 * T * tokens * case["Hq"] * D}
    moved = B * ((T - 1) // 2 + 1) / 2  # half the longest accepted path on average
    return {"bytes": 2 * 2 * 2 * moved * Hkv * D, "flops": 0}


# ---- in 64 bits, from the definitions ---------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "keep":
        return None  # values are moved, not computed
    if case["op"] == "sample":
        return {"token": None, "prob": _exact_prob(s)}
    B, T, Hkv, D, page = case["B"], case["T"], case["Hkv"], case["D"], case["page"]
    lens = [int(n) for n in s["len"]]
    if case["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=k.device)
        spin = torch.exp(-2.0 * i / case["rot"] * math.log(THETA))
        first, second = (2 * i.long(), 2 * i.long() + 1) if case["pairs"] else (i.long(), i.long() + case["rot"] // 2)

        def turned(x, gamma, at):  # x [T, H, D]
            x = x.double()
            x = x * gamma.double() * torch.rsqrt((x * x).sum(-1, keepdim=True) / D + EPS)
            z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(spin), at[:, None] * spin)[:, None]
            x[..., first], x[..., second] = z.real, z.imag
            return x

        q = torch.empty(B * T, case["Hq"] * D, dtype=torch.float64, device=k.device)
        for b, n in enumerate(lens):
            rows = slice(b * T, (b + 1) * T)
            at = n + (s["depth"].double() if s["depth"] is not None else torch.arange(T, dtype=torch.float64, device=k.device))
            q[rows] = turned(s["q_in"][rows].view(T, -1, D), s["q_gamma"], at).flatten(1)
            kk = turned(s["k_in"][rows].view(T, -1, D), s["k_gamma"], at)
            vv = s["v_in"][rows].view(T, -1, D).double()
            place = torch.arange(n, n + T, device=k.device)
            where = s["table"][b].long()[place // page]
            k[where, :, place % page], v[where, :, place % page] = kk, vv
        return {"q": q, "k": k, "v": v}
    g = case["Hq"] // Hkv
    out = torch.empty(B * T, case["Hq"], D, dtype=torch.float64, device=s["q"].device)
    mask = [int(m) for m in s["mask"]]
    for b, n in enumerate(lens):
        used = s["table"][b, : -(-(n + T) // page)].long()
        open_ = torch.ones(T, n + T, dtype=torch.bool, device=out.device)
        open_[:, n:] = torch.tensor([[mask[t] >> j & 1 == 1 for j in range(T)] for t in range(T)], device=out.device)
        for h in range(Hkv):
            kk = s["k"][used, h].double().reshape(-1, D)[: n + T]
            vv = s["v"][used, h].double().reshape(-1, D)[: n + T]
            qq = s["q"][b * T:(b + 1) * T].double().view(T, -1, D)[:, h * g:(h + 1) * g]
            e = torch.einsum("tgd,nd->tgn", qq, kk) / math.sqrt(D)
            e = torch.softmax(e.masked_fill(~open_[:, None], -math.inf), -1)
            out[b * T:(b + 1) * T, h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", e, vv)
    return out.reshape(B * T, -1)


def _exact_prob(s):
    """The chosen tokens' probabilities, row by row."""
    host = {n: None if s[n] is None else s[n].double().cpu().numpy() for n in ("logits", "u", "temperature", "top_k", "top_p", "min_p")}
    probs = []
    for m, x in enumerate(host["logits"]):
        if host["temperature"][m] <= 0:
            probs.append(1.0)
            continue
        order = np.argsort(-x, kind="stable")
        w = np.exp((x[order] - x[order[0]]) / host["temperature"][m])
        n = len(w)
        if host["top_k"] is not None:
            n = min(n, int(host["top_k"][m]))
        if host["top_p"] is not None:
            sums = np.cumsum(w[:n])
            n = 1 + int(np.searchsorted(sums[:-1], host["top_p"][m] * sums[-1], side="left"))
        if host["min_p"] is not None:
            n = int(np.count_nonzero(w[:n] >= host["min_p"][m]))
        index = np.sort(order[:n])
        w = np.exp((x[index] - x[order[0]]) / host["temperature"][m])
        sums = np.cumsum(w)
        at = min(int(np.searchsorted(sums, host["u"][m] * sums[-1], side="right")), n - 1)
        probs.append(w[at] / sums[-1])
    return torch.tensor(probs, dtype=torch.float64)
