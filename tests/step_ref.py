"""Plain 64-bit forms of the step operators, on the CPU, row by row, and the
error bounds of the kernels' arithmetic against them."""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative


def rows_in_use(step_len, count, T, b):
    if step_len[b] < 0:
        return 0
    return T if count is None else max(0, min(T, int(count[b])))


def append_row(x, gamma, eps, pos, radians, pairs):
    """x [H, D] in 64 bits -> the normed and rotated row."""
    x = x.double()
    if gamma is not None:
        x = x * gamma.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = len(radians)
    out = x.clone()
    for i, f in enumerate(radians):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + n)
        # the angle modulo a turn, reduced in integers as far as the 53-bit frequency goes
        ang = math.fmod(pos * f, 2 * math.pi)
        c, s = math.cos(ang), math.sin(ang)
        out[:, a] = x[:, a] * c - x[:, b] * s
        out[:, b] = x[:, b] * c + x[:, a] * s
    return out


def append_bound(ref, dtype):
    """Half a step of the result's type, and the fp32 arithmetic before it, in
    units of 2^-24 of the head's largest value m (a rotated pair reaches 2 m):
    the norm at most D/32 + 9 roundings of the sum of squares, halved by the
    root, and 4 more factors: 17 / 2 + 4 <= 13; the angle's last conversion
    (pi 2^-25) and sincospi (2 ulp): 4; product and sum: 3.  20 * 2 m.  fp16
    results below 2^-14 step by 2^-24."""
    m = ref.abs().amax(-1, keepdim=True)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return HALF[dtype] * ref.abs() + 40 * 2.0 ** -24 * m * (1 + HALF[dtype]) + tiny


def attention_rows(q, k, v, seen, scale):
    """q [R, D], k and v [N, D], seen [R, N]: the rows' results in 64 bits, the
    weights' mean of |v| and of nothing else, and the scores' error unit."""
    q, k, v = q.double(), k.double(), v.double()
    used = seen.any(0)
    k, v = torch.where(used[:, None], k, 0), torch.where(used[:, None], v, 0)
    s = (q @ k.T) * scale
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    w = torch.where(seen, torch.exp(s - torch.where(m > -math.inf, m, 0)), 0)
    l = w.sum(-1, keepdim=True)
    p = torch.where(l > 0, w / l, 0)
    size = (q.abs() @ k.abs().T).masked_fill(~seen, 0).amax(-1, keepdim=True) * abs(scale)
    return p @ v, p @ v.abs(), size, (seen.double() @ v.abs()) / torch.where(l > 0, l, 1)


def attention_bound(o, a, size, mass, D, dtype):
    """a = sum_j p_j |v_j|.  The output's rounding to bf16, half a step of |o|.
    The weights' rounding to the cache's type: half a step of a.  A score's
    error d = (D + 8) 2^-24 sum |q||k| scale (fp32 dot product, scale folded
    into log2 units) moves every weight by at most 2 d relative, as 2^x and the
    fp32 sums (2^-20 together) do.  fp16 weights below 2^-14 of the row's
    largest step by 2^-24: 2^-25 of sum |v_j| / l."""
    d = (D + 8) * 2.0 ** -24 * size
    low = 2.0 ** -25 * mass if dtype == torch.float16 else 0.0
    return 2.0 ** -8 * o.abs() + (1 + 2.0 ** -8) * ((HALF[dtype] + 2 * d + 2.0 ** -20) * a + low) + 1e-30


def sample_row(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability) of one row of logits (float64 numpy), by sorting."""
    V = len(x)
    if np.isnan(x).any() or np.all(x == -np.inf):
        return -1, 0.0
    if not temperature > 0:
        return int(np.argmax(x)), 1.0
    if np.max(x) == np.inf:
        x = np.where(x == np.inf, 0.0, -np.inf)
    order = np.lexsort((np.arange(V), -x))
    w = np.exp((x[order] - x[order[0]]) / temperature)
    n = V if not 0 < top_k < V else top_k
    if top_p < 1:
        share = max(top_p, 0) * math.fsum(w[:n])
        before, keep = 0.0, 0
        sums = np.concatenate([[0.0], np.cumsum(w[:n])])
        while keep < n and (keep == 0 or sums[keep] < share):
            keep += 1
        n = keep
    kept = np.zeros(V, bool)
    kept[order[:n]] = w[:n] >= (min(min_p, 1.0) if min_p > 0 else 0.0)
    weight = np.zeros(V)
    weight[order] = w
    weight[~kept] = 0.0
    weight[weight < 2.0 ** -43] = 0.0  # weights are multiples of 2^-42 (half units round up): these are none
    total = math.fsum(weight)
    sums = np.cumsum(weight)
    alive = np.nonzero(weight > 0)[0]
    past = alive[sums[alive] > min(max(u, 0.0), 1.0) * total]
    token = int(past[0]) if len(past) else int(alive[-1])
    return token, float(weight[token] / total)
