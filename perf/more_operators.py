"""Operators around the paged cache and the logits of a decode / verification step: what is measured of them.

Four operators: ``kv_append`` with positions of several axes (the rows of an image or a video, and rows whose place in the
cache is not their position), ``kv_weigh`` (the attention weight that each cached token got from a step's rows, accumulated),
``kv_evict`` (the tokens of least accumulated weight leave the cache, head by head) and ``adjust_logits`` (penalties for
repeated tokens, biases and grammar masks).  ``run`` computes them in plain torch operations, or, where ``own`` is true, by
the framework's calls; ``exact`` in 64 bits.
"""
import math

import torch

own = False

THETA = 1.0e6   # base of the rotation's frequencies
EPS = 1.0e-6    # of the norms
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # the projections of one decoded token behind an image: the smallest append
        dict(name="append_token", op="append", B=1, T=1, Hq=24, Hkv=4, D=256, rot=64, pairs=False, dealt=True, src="f32",
             cache="bf16", page=64, len=2000),
        # the rows of one image and the text around it, an odd number of them, from a bf16 projection
        dict(name="append_image", op="append", B=1, T=2411, Hq=24, Hkv=4, D=256, rot=64, pairs=False, dealt=True, src="bf16",
             cache="bf16", page=64, len=77),
        # two videos' rows, whole heads turning, pairs side by side, axes one behind the other
        dict(name="append_video", op="append", B=2, T=2049, Hq=48, Hkv=8, D=128, rot=128, pairs=True, dealt=False, src="f32",
             cache="f16", page=32, len=517),
        # one token's weights over a short chat
        dict(name="weigh_token", op="weigh", B=1, T=1, Hq=24, Hkv=4, D=256, cache="bf16", page=64, len=1777, path=False, decay=1.0),
        # the accepted paths of several requests of different lengths, five rows each, older weights fading
        dict(name="weigh_batch", op="weigh", B=8, T=5, Hq=48, Hkv=8, D=128, cache="f16", page=32, len=30011, path=True, decay=0.97),
        # the last rows of a book's prompt look back over it: the largest cache and 96 query rows per cache head
        dict(name="weigh_window", op="weigh", B=1, T=16, Hq=48, Hkv=8, D=128, cache="bf16", page=16, len=130999, path=False, decay=1.0),
        # while decoding: a few dozen tokens over the room
        dict(name="evict_few", op="evict", B=1, Hkv=8, D=128, cache="bf16", page=16, len=4130, keep=0.99, recent=128, moved=True),
        # a long prompt cut to an eighth
        dict(name="evict_prompt", op="evict", B=1, Hkv=4, D=256, cache="bf16", page=64, len=131000, keep=0.125, recent=512, moved=False),
        # a batch of different lengths halved
        dict(name="evict_batch", op="evict", B=16, Hkv=8, D=128, cache="f16", page=32, len=9001, keep=0.5, recent=64, moved=True),
        # one row of a small vocabulary, a short history
        dict(name="adjust_token", op="adjust", B=1, T=1, V=32000, dtype="f32", history=311, bias=0, allowed=0.0),
        # every row of a tree, a long history, biases, a grammar that leaves a third of an odd vocabulary
        dict(name="adjust_tree", op="adjust", B=1, T=8, V=131071, dtype="f32", history=20011, bias=64, allowed=0.33),
        # a large batch of 16-bit logits over a large vocabulary
        dict(name="adjust_batch", op="adjust", B=64, T=1, V=262144, dtype="bf16", history=4096, bias=16, allowed=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "weigh", "weigh", "evict", "evict", "adjust", "adjust"])
    if op == "adjust":
        T = rng.choice([1, 1, 2, 5, 8])
        return dict(op=op, B=_log_int(rng, 1, 64 // T), T=T, V=_log_int(rng, 500, 262144), dtype=rng.choice(["f32", "bf16"]),
                    history=_log_int(rng, 1, 60000) if rng.random() < 0.3 else _log_int(rng, 1, 5000),
                    bias=rng.choice([0, 1, 20, 300]), allowed=rng.choice([0.0, 0.001, 0.33, 0.9]))
    D, Hkv = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 5, 8])
    case = dict(op=op, B=1, T=1, Hkv=Hkv, D=D, cache=rng.choice(["bf16", "f16"]), page=rng.choice([16, 32, 64, 128]), len=0)
    if op == "append":
        case["Hq"] = Hkv * rng.choice([1, 2, 3, 6, 8])
        case["rot"] = rng.choice([D, D // 2, D // 4])
        case["pairs"], case["dealt"] = rng.random() < 0.5, rng.random() < 0.5
        case["src"] = rng.choice(["f32", "bf16"])
        case["T"] = _log_int(rng, 1, 2000)
        case["B"] = rng.choice([1, 1, 2, 3]) if case["T"] > 32 else rng.choice([1, 1, 2, 8, 13])
        case["len"] = _log_int(rng, 1, 60000 // case["B"])
    elif op == "weigh":
        g = rng.choice([1, 2, 3, 6, 8])
        case["Hq"] = Hkv * g
        case["T"] = rng.choice([1, 1, 2, 3, 5, 8, 8, 16])
        case["B"] = rng.choice([1, 1, 1, 2, 5, 8, 19])
        case["len"] = _log_int(rng, 1, 131000 * 1024 // (Hkv * D) // case["B"] // (1 + case["T"] // 16))
        case["len"] = max(1, min(case["len"], 200000))
        case["path"], case["decay"] = rng.random() < 0.5, rng.choice([1.0, 0.97, 0.5])
    else:
        del case["T"]
        case["B"] = rng.choice([1, 1, 2, 5, 16])
        case["len"] = _log_int(rng, 1, max(2, min(131000, 131000 * 1024 // (Hkv * D) // case["B"])))
        case["keep"], case["recent"] = rng.choice([0.03, 0.125, 0.5, 0.9, 0.99, 1.0]), rng.choice([0, 16, 256])
        case["moved"] = rng.random() < 0.5
    return case


def _lens(case):
    """The sequences' committed tokens: the first the longest, down to a quarter of it."""
    B, n = case["B"], case["len"]
    return [max(1, n - (3 * n * b) // (4 * B)) for b in range(B)]


def _tree(T):
    """Parents of a drafted tree's rows: row 0 the committed token, then two branches, each a chain."""
    half = 1 + (T - 1 + 1) // 2
    return [-1] + [0 if t in (1, half) else t - 1 for t in range(1, T)]


def _branch(T):
    """A drafted tree's second branch, which is accepted up to some length: row 0 and the rows behind the first branch."""
    second = 1 + T // 2
    return [0] + list(range(second, T)) if T > 2 else list(range(T))


def _sections(n):
    """Pairs of the time, height and width axes: nearly a third each."""
    return [n - 2 * (n // 3), n // 3, n // 3]


def _axes(n, dealt):
    """The axis of each pair: the sections one behind the other, or dealt in turn to the axes that still have some."""
    left = _sections(n)
    if not dealt:
        return [a for a in range(3) for _ in range(left[a])]
    axis = []
    while len(axis) < n:
        for a in range(3):
            if left[a]:
                left[a] -= 1
                axis.append(a)
    return axis


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"op": case["op"], "case": case}
    if case["op"] == "adjust":
        _prepare_adjust(s, case, dev, g)
        return s
    B, Hkv, D, page, dt = case["B"], case["Hkv"], case["D"], case["page"], DTYPES[case["cache"]]
    T = case.get("T", 1)
    per = -(-(case["len"] + T) // page)
    pages = B * per + 3
    s["k"] = torch.randn(pages, Hkv, page, D, device=dev, generator=g, dtype=dt)
    s["v"] = torch.randn(pages, Hkv, page, D, device=dev, generator=g, dtype=dt)
    s["table"] = torch.randperm(pages, device=dev, generator=g)[: B * per].view(B, per).to(torch.int32)
    s["len"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
    s["depth"] = s["mask"] = None
    if case["op"] == "append":
        src, Hq, n = DTYPES[case["src"]], case["Hq"], B * T
        s["q_in"] = torch.randn(n, Hq * D, device=dev, generator=g).mul_(1.7).to(src)
        s["k_in"] = torch.randn(n, Hkv * D, device=dev, generator=g).mul_(2.3).to(src)
        s["v_in"] = torch.randn(n, Hkv * D, device=dev, generator=g).to(src)
        s["q_gamma"] = 0.5 + torch.rand(D, device=dev, generator=g)
        s["k_gamma"] = 0.5 + torch.rand(D, device=dev, generator=g)
        s["q"] = torch.empty(n, Hq * D, dtype=dt, device=dev)
        # frames of a grid, row by row, behind a text as long as the committed tokens
        side = max(1, int(math.sqrt(T / 3)))
        i = torch.arange(T, device=dev)
        grid = torch.stack([i // (side * side), i // side % side, i % side], 1)
        s["position"] = (s["len"].long()[:, None, None] + grid).reshape(n, 3).to(torch.int32)
    else:
        room = case["len"] + T + 5
        s["score"] = torch.rand(B, Hkv, room, device=dev, generator=g).log_().neg_().pow_(3)  # few tokens hold most of it
        s["score_out"] = torch.zeros(B, Hkv, room, device=dev)
        s["position"] = torch.arange(room, device=dev, dtype=torch.int32).repeat(B, Hkv, 1)
    if case["op"] == "weigh":
        _prepare_weigh(s, case, dev, g)
    elif case["op"] == "evict":
        lens = s["len"].long()
        s["n_keep"] = (lens.double() * case["keep"]).long().clamp(min=1).to(torch.int32)
        s["since"] = (lens - case["recent"]).to(torch.int32)
        s["first"] = 4
        s["len_out"] = torch.empty(B, dtype=torch.int32, device=dev)
        if case["moved"]:  # an earlier eviction has moved tokens: places are not positions
            shuffled = torch.rand(B, Hkv, room, device=dev, generator=g)
            shuffled.masked_fill_(torch.arange(room, device=dev) >= lens[:, None, None], 2.0)
            s["position"] = shuffled.argsort(-1).to(torch.int32)
        else:
            s["position"] = None
        s["position_out"] = torch.zeros(B, Hkv, room, dtype=torch.int32, device=dev)
    if own:
        from w6a8_quantized_linear_gb300 import qlin
        s["cache"] = qlin.KVCache(s["k"], s["v"])
        s["step"] = qlin.KVStep(s["table"], s["len"], T, depth=s["depth"], mask=s["mask"])
        if case["op"] == "append":
            s["turns"] = qlin.rope_turns(THETA, case["rot"], device=dev)
            s["axis"] = qlin.rope_axes(_sections(case["rot"] // 2), dealt=case["dealt"])
        elif case["op"] == "evict":
            s["ws"] = qlin.new_workspace(qlin.kv_evict_workspace_bytes(s["cache"], s["step"], room), dev)
    return s


def _prepare_weigh(s, case, dev, g):
    """A step that has gone through attention: its rows' softmax statistics, and which of them were accepted."""
    B, T, Hq, Hkv, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]
    s["q"] = torch.randn(B * T, Hq * D, device=dev, generator=g).to(DTYPES[case["cache"]])
    if case["path"]:
        parent, mask = _tree(T), [1]
        for t in range(1, T):
            mask.append(mask[parent[t]] | 1 << t)
        s["mask"] = torch.tensor(mask, dtype=torch.int32, device=dev)
        path = _branch(T)
        s["keep"] = torch.tensor([path + [0] * (T - len(path))] * B, dtype=torch.int32, device=dev)
        s["n_keep"] = torch.randint(1, len(path) + 1, (B,), device=dev, generator=g, dtype=torch.int32)
    else:  # rows that follow one another, all of them kept
        mask = [(2 << t) - 1 for t in range(T)]
        s["keep"] = s["n_keep"] = None
    s["at"] = (s["len"].long()[:, None] + torch.arange(T, device=dev)).flatten().to(torch.int32)
    s["position_out"] = torch.zeros(B, Hkv, s["score"].shape[2], dtype=torch.int32, device=dev)
    stats = torch.empty(B * T, Hq, 2, device=dev)  # as attention gives them: a reference in log2 units, the sum of 2^(x - it)
    open_ = torch.tensor([[m >> j & 1 == 1 for j in range(T)] for m in mask], device=dev)
    for b, n in enumerate(_lens(case)):
        seen = torch.cat([torch.ones(T, n, dtype=torch.bool, device=dev), open_], 1)
        k = s["k"][s["table"][b].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, : n + T]
        for h in range(Hkv):
            q = s["q"][b * T:(b + 1) * T].view(T, Hkv, -1, D)[:, h].float()
            x = (q @ k[h].float().t()) * (D ** -0.5 * math.log2(math.e))
            x = x.masked_fill(~seen[:, None], -math.inf)
            r = x.amax(-1)
            rows = stats[b * T:(b + 1) * T].view(T, Hkv, -1, 2)[:, h]
            rows[..., 0], rows[..., 1] = r, torch.exp2(x - r[..., None]).sum(-1)
    s["stats"] = stats


def _prepare_adjust(s, case, dev, g):
    B, T, V, L = case["B"], case["T"], case["V"], case["history"]
    s["logits"] = (torch.randn(B * T, V, device=dev, generator=g) * 2.5).to(DTYPES[case["dtype"]])
    s["out"] = torch.empty_like(s["logits"])
    # few tokens make up most of a text
    s["history"] = (torch.rand(B, L, device=dev, generator=g).pow(5) * V).long().clamp(max=V - 1).to(torch.int32)
    s["history_len"] = torch.tensor([max(1, L - (L * b) // (2 * B)) for b in range(B)], dtype=torch.int32, device=dev)
    s["prompt_len"] = s["history_len"] // 3
    s["repetition"] = 1.0 + 0.3 * torch.rand(B, device=dev, generator=g)
    s["presence"] = 0.5 * torch.rand(B, device=dev, generator=g)
    s["frequency"] = 0.2 * torch.rand(B, device=dev, generator=g)
    s["draft"] = s["mask"] = None
    if T > 1:
        parent, mask = _tree(T), [1]
        for t in range(1, T):
            mask.append(mask[parent[t]] | 1 << t)
        s["mask"] = torch.tensor(mask, dtype=torch.int32, device=dev)
        s["draft"] = (torch.rand(B, T, device=dev, generator=g).pow(5) * V).long().clamp(max=V - 1).to(torch.int32)
    s["bias_token"] = s["bias"] = s["allowed"] = None
    n = min(case["bias"], V)
    if n:
        s["bias_token"] = torch.stack([torch.randperm(V, device=dev, generator=g)[:n] for _ in range(B)]).to(torch.int32)
        s["bias"] = 4 * torch.randn(B, n, device=dev, generator=g)
    if case["allowed"]:
        words = -(-V // 32)
        bits = torch.rand(B * T, words, 32, device=dev, generator=g) < case["allowed"]
        bits = (bits.long() << torch.arange(32, device=dev)).sum(-1)
        s["allowed"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)


# ---- the plain forms ------------------------------------------------------------------------------------------------

def _places(s, at):
    """Page and row in the page of the tokens at [B, ...]."""
    page = s["case"]["page"]
    return s["table"].long().gather(1, (at // page).flatten(1)).view(at.shape), at % page


def _plain_append(s):
    c = s["case"]
    B, T, D, dt, rot = c["B"], c["T"], c["D"], DTYPES[c["cache"]], c["rot"]
    freq = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=s["len"].device) / rot)
    axis = torch.tensor(_axes(rot // 2, c["dealt"]), device=s["len"].device)
    angle = s["position"].double()[:, axis] * freq  # in 64 bits: far positions
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, gamma):
        x = x.view(B * T, -1, D).float()
        x = x * gamma / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        head, rest = x[..., :rot], x[..., rot:]
        if c["pairs"]:
            a, b = head[..., 0::2], head[..., 1::2]
            return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)

    q, k = turned(s["q_in"], s["q_gamma"]), turned(s["k_in"], s["k_gamma"])
    p, r = _places(s, s["len"].long()[:, None] + torch.arange(T, device=q.device))
    s["k"][p.flatten(), :, r.flatten()] = k.to(dt)
    s["v"][p.flatten(), :, r.flatten()] = s["v_in"].view(B * T, -1, D).to(dt)
    return {"q": q.reshape(B * T, -1).to(dt), "k": s["k"], "v": s["v"]}


def _plain_weigh(s):
    c = s["case"]
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    g, room, dev = Hq // Hkv, s["score"].shape[2], s["q"].device
    i = torch.arange(T, device=dev)
    keep = i.repeat(B, 1) if s["keep"] is None else s["keep"].long()
    n_keep = torch.full((B,), T, device=dev) if s["n_keep"] is None else s["n_keep"].long()
    there = i < n_keep[:, None]                                    # [B, T], of the kept rows
    base = s["len"].long()[:, None]
    token = torch.arange(room, device=dev)
    old = token < base                                             # [B, room], committed
    # the tokens' keys: the committed ones where they lie, then the kept rows' in order
    at = torch.arange(room - 5, device=dev).repeat(B, 1)
    k = s["k"][s["table"].long()].transpose(1, 2).reshape(B, Hkv, -1, D)
    place = at.scatter(1, torch.where(there, base + i, at[:, :T]), torch.where(there, base + keep, at[:, :T]))
    k = k.gather(2, place[:, None, :, None].expand(B, Hkv, -1, D)).float()
    rows = torch.arange(B, device=dev)[:, None] * T + keep         # [B, T], kept rows among all
    q = s["q"].view(B * T, Hkv, g, D)[rows].permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * g, D).float()
    r, l = s["stats"].view(B * T, Hkv, g, 2)[rows].permute(4, 0, 2, 1, 3).reshape(2, B, Hkv, T * g, 1)
    x = (q @ k.transpose(-1, -2)) * (D ** -0.5 * math.log2(math.e))
    w = torch.exp2(x - r) / l
    seen = there[:, :, None] & (at[:, None] <= base[:, None] + i[:, None])  # row i sees the committed tokens and rows 0 .. i
    w = torch.where(seen[:, None, :, None], w.view(B, Hkv, T, g, -1), 0.0).sum((2, 3))
    new = (token >= base) & (token < base + n_keep[:, None])
    w = torch.nn.functional.pad(w, (0, 5))
    score = torch.where(old[:, None], c["decay"] * s["score"] + w, w)
    s["score_out"].copy_(torch.where((old | new)[:, None], score, s["score_out"]))
    where = s["at"].long()[rows].gather(1, (token - base).clamp(0, T - 1)).to(torch.int32)
    s["position_out"].copy_(torch.where(new[:, None], where[:, None], s["position_out"]))
    return {"score": s["score_out"], "position": s["position_out"]}


def _plain_evict(s):
    B, H, room = s["score"].shape
    i = torch.arange(room, device=s["score"].device)
    n, n_keep = s["len"].long()[:, None, None], s["n_keep"].long()[:, None, None]
    position = i.to(torch.int32).expand(B, H, room) if s["position"] is None else s["position"]
    safe = (position < s["first"]) | (position >= s["since"][:, None, None])
    key = torch.where(safe, math.inf, s["score"])
    key = torch.where(i < n, key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, i.expand(B, H, room))
    stays = torch.minimum(n, n_keep)
    kept = (rank < stays) & (i < n)
    score, moved = s["score_out"], s["position_out"]
    low = kept & (i < stays)
    score.copy_(torch.where(low, s["score"], score))
    moved.copy_(torch.where(low, position, moved))
    b, h, to = (~kept & (i < stays)).nonzero(as_tuple=True)  # as many holes as tokens behind them, item by item
    _, _, of = (kept & (i >= stays)).nonzero(as_tuple=True)
    score[b, h, to], moved[b, h, to] = s["score"][b, h, of], position[b, h, of]
    page = s["case"]["page"]
    table = s["table"].long()
    for x in (s["k"], s["v"]):
        x[table[b, to // page], h, to % page] = x[table[b, of // page], h, of % page]
    return {"k": s["k"], "v": s["v"], "score": score, "position": moved, "len": stays.flatten().to(torch.int32)}


def _plain_adjust(s):
    c = s["case"]
    B, T, V, L = c["B"], c["T"], c["V"], c["history"]
    dev = s["logits"].device
    x = s["logits"].float().view(B, T, V)
    i = torch.arange(L, device=dev)
    there, output = i < s["history_len"][:, None], i >= s["prompt_len"][:, None]
    tokens = s["history"].long()
    seen = torch.zeros(B, V, dtype=torch.int32, device=dev).scatter_add_(1, tokens, there.int())
    count = torch.zeros(B, V, dtype=torch.int32, device=dev).scatter_add_(1, tokens, (there & output).int())
    seen, count = seen[:, None].repeat(1, T, 1), count[:, None].repeat(1, T, 1)
    if s["draft"] is not None:
        path = (s["mask"].long()[:, None] >> torch.arange(T, device=dev) & 1).int().expand(B, T, T)
        index = s["draft"].long()[:, None].expand(B, T, T)
        seen.scatter_add_(2, index, path)
        count.scatter_add_(2, index, path)
    r, p, f = (s[name][:, None, None] for name in ("repetition", "presence", "frequency"))
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = torch.where(count > 0, x - f * count - p, x)
    if s["bias"] is not None:
        x = x.scatter_add(2, s["bias_token"].long()[:, None].expand(B, T, -1), s["bias"][:, None].expand(B, T, -1))
    x = x.view(B * T, V)
    if s["allowed"] is not None:
        v = torch.arange(V, device=dev)
        x = torch.where((s["allowed"][:, v // 32] >> (v % 32).int()) & 1 == 1, x, -math.inf)
    s["out"].copy_(x)
    return s["out"]


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return {"append": _plain_append, "weigh": _plain_weigh, "evict": _plain_evict, "adjust": _plain_adjust}[s["op"]](s)
    from w6a8_quantized_linear_gb300 import qlin
    c = s["case"]
    if s["op"] == "append":
        qlin.kv_append(s["cache"], s["step"], q=s["q_in"], k=s["k_in"], v=s["v_in"], q_gamma=s["q_gamma"], k_gamma=s["k_gamma"],
                       eps=EPS, turns=s["turns"], pairs=c["pairs"], q_out=s["q"], position=s["position"], axis=s["axis"])
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    if s["op"] == "weigh":
        qlin.kv_weigh(s["cache"], s["step"], s["q"], s["stats"], s["score"], keep=s["keep"], n_keep=s["n_keep"], decay=c["decay"],
                      score_out=s["score_out"], position_out=s["position_out"], at=s["at"])
        return {"score": s["score_out"], "position": s["position_out"]}
    if s["op"] == "evict":
        qlin.kv_evict(s["cache"], s["step"], s["score"], s["n_keep"], first=s["first"], since=s["since"], position=s["position"],
                      score_out=s["score_out"], position_out=s["position_out"], len_out=s["len_out"], ws=s["ws"])
        return {"k": s["k"], "v": s["v"], "score": s["score_out"], "position": s["position_out"], "len": s["len_out"]}
    return qlin.adjust_logits(s["logits"], out=s["out"], history=s["history"], history_len=s["history_len"],
                              prompt_len=s["prompt_len"], draft=s["draft"], mask=s["mask"], repetition=s["repetition"],
                              presence=s["presence"], frequency=s["frequency"], bias_token=s["bias_token"], bias=s["bias"],
                              allowed=s["allowed"])


def work(case):
    if case["op"] == "adjust":
        B, T, V = case["B"], case["T"], case["V"]
        n = B * T * V
        words = B * T * -(-V // 32) if case["allowed"] else 0
        return {"bytes": 2 * n * (4 if case["dtype"] == "f32" else 2) + 4 * words + 3 * B * case["history"], "flops": 0}
    Hkv, D = case["Hkv"], case["D"]
    tokens = sum(_lens(case))
    if case["op"] == "append":
        n = case["B"] * case["T"]
        values = n * (case["Hq"] + 2 * Hkv) * D
        return {"bytes": values * ((4 if case["src"] == "f32" else 2) + 2) + 12 * n, "flops": 8 * n * (case["Hq"] + Hkv) * D}
    if case["op"] == "weigh":
        n = case["B"] * case["T"]
        return {"bytes": (2 * D + 8) * tokens * Hkv + 2 * n * (Hkv + case["Hq"]) * D + 8 * n * case["Hq"],
                "flops": 2 * case["T"] * tokens * case["Hq"] * D}
    kept = sum(max(1, int(n * case["keep"])) for n in _lens(case))
    moved = kept * (1 - kept / tokens)  # the kept ones that lie behind the places left, where weights are spread evenly
    per = 4 if case["moved"] else 0
    return {"bytes": Hkv * ((4 + per) * tokens + 8 * kept + 2 * 2 * 2 * D * moved), "flops": 0}


# ---- in 64 bits, from the definitions ---------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "evict":
        return None  # values are moved, not computed
    s = prepare(case, seed)
    return {"append": _exact_append, "weigh": _exact_weigh, "adjust": _exact_adjust}[case["op"]](s, case)


def _exact_append(s, case):
    B, T, D, page, rot = case["B"], case["T"], case["D"], case["page"], case["rot"]
    k, v = s["k"].double(), s["v"].double()
    half = rot // 2
    first = [2 * i if case["pairs"] else i for i in range(half)]
    second = [2 * i + 1 if case["pairs"] else i + half for i in range(half)]
    axis, spin = _axes(half, case["dealt"]), [math.exp(-2.0 * i / rot * math.log(THETA)) for i in range(half)]
    spin = torch.tensor(spin, dtype=torch.float64, device=k.device)
    phase = torch.polar(torch.ones_like(spin), torch.stack([s["position"][:, a].double() for a in axis], 1) * spin)

    def turned(x, gamma, rows):
        x = x[rows].reshape(T, -1, D).double()
        x = x * gamma.double() * torch.rsqrt((x * x).sum(-1, keepdim=True) / D + EPS)
        z = torch.complex(x[..., first], x[..., second]) * phase[rows][:, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q = torch.empty(B * T, case["Hq"] * D, dtype=torch.float64, device=k.device)
    for b, n in enumerate(_lens(case)):
        rows = slice(b * T, (b + 1) * T)
        q[rows] = turned(s["q_in"], s["q_gamma"], rows).flatten(1)
        at = torch.arange(n, n + T, device=k.device)
        where = s["table"][b].long()[at // page]
        k[where, :, at % page] = turned(s["k_in"], s["k_gamma"], rows)
        v[where, :, at % page] = s["v_in"][rows].view(T, -1, D).double()
    return {"q": q, "k": k, "v": v}


def _exact_weigh(s, case):
    B, T, Hkv, D, page = case["B"], case["T"], case["Hkv"], case["D"], case["page"]
    out = s["score_out"].double()
    for b, n in enumerate(_lens(case)):
        path = list(range(T)) if s["keep"] is None else s["keep"][b, : int(s["n_keep"][b])].tolist()
        tokens = torch.cat([torch.arange(n, device=out.device), n + torch.tensor(path, device=out.device)])
        where = s["table"][b].long()[tokens // page]
        for h in range(Hkv):
            k = s["k"][where, h, tokens % page].double()
            total = torch.zeros(n + len(path), dtype=torch.float64, device=out.device)
            for i, t in enumerate(path):
                q = s["q"][b * T + t].double().view(Hkv, -1, D)[h]
                stat = s["stats"][b * T + t].double().view(Hkv, -1, 2)[h]
                e = torch.exp(math.log(2.0) * (k[: n + i + 1] @ q.t() * (math.log2(math.e) / math.sqrt(D)) - stat[:, 0]))
                total[: n + i + 1] += (e / stat[:, 1]).sum(1)
            total[:n] += case["decay"] * s["score"][b, h, :n].double()
            out[b, h, : n + len(path)] = total
    return {"score": out, "position": None}


def _exact_adjust(s, case):
    B, T, V = case["B"], case["T"], case["V"]
    out = s["logits"].double()
    for b in range(B):
        n, first = int(s["history_len"][b]), int(s["prompt_len"][b])
        for t in range(T):
            x = out[b * T + t]
            path = s["history"][b, :0].long()
            if s["draft"] is not None:
                bits = int(s["mask"][t])
                path = s["draft"][b, [j for j in range(T) if bits >> j & 1]].long()
            all_ = torch.cat([s["history"][b, :n].long(), path])
            made = torch.cat([s["history"][b, first:n].long(), path])
            token = torch.unique(all_)
            r = s["repetition"][b].double()
            x[token] = torch.where(x[token] > 0, x[token] / r, x[token] * r)
            token, times = torch.unique(made, return_counts=True)
            x[token] -= s["frequency"][b].double() * times + s["presence"][b].double()
            if s["bias"] is not None:
                x[s["bias_token"][b].long()] += s["bias"][b].double()
            if s["allowed"] is not None:
                word = s["allowed"][b * T + t].long() & 0xFFFFFFFF
                bits = (word[:, None] >> torch.arange(32, device=word.device) & 1).flatten()[:V]
                x[bits == 0] = -math.inf
    return out
