"""Plain 64-bit implementations (on the host) of the expert operators and of the
products in 8-bit integers, one value at a time where that keeps them plain, and
the bounds that the tests hold the kernels to.

Rounding to a type is off by at most half a step, U of the value: 2^-24 for
float32, 2^-8 for bfloat16."""

from __future__ import annotations

import math

import numpy as np
import torch

U32, U = 2.0 ** -24, {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BOTH = (torch.float32, torch.bfloat16)


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32)


def scores(l, score):
    """l: list of floats of one token -> scores in 64 bits (masked experts: None)."""
    live = [x != -math.inf for x in l]
    if score == "sigmoid":
        return [(1 / (1 + math.exp(-x)) if x > -700 else math.exp(x)) if ok else None for x, ok in zip(l, live)]
    top = max((x for x, ok in zip(l, live) if ok), default=0.0)
    e = [math.exp(x - top) if ok else 0.0 for x, ok in zip(l, live)]
    return [x / sum(e) if ok else None for x, ok in zip(e, live)]


def choose(l, k, score="softmax", bias=None, groups=1, top_groups=1, group_score="max"):
    """The experts of one token, best first, -1 where none is left."""
    s = scores(l, score)
    c = [None if x is None else x + (0.0 if bias is None else bias[i]) for i, x in enumerate(s)]
    c = [None if x == -math.inf else x for x in c]
    order = c if bias is not None else [None if x is None else l[i] for i, x in enumerate(c)]
    allowed = range(len(l))
    if groups > 1:
        size = len(l) // groups
        rated = []
        for g in range(groups):
            mine = range(g * size, (g + 1) * size)
            best = sorted((c[i] for i in mine if c[i] is not None), reverse=True)
            if group_score == "max":
                by = max((order[i] for i in mine if order[i] is not None), default=None)
            else:
                by = sum(best[:2]) if best else None
            rated.append((-math.inf if by is None else by, -g, by is not None))
        kept = sorted(rated, reverse=True)[:top_groups]
        allowed = [i for _, g, some in kept if some for i in range(-g * size, (-g + 1) * size)]
    ranked = sorted((i for i in allowed if order[i] is not None), key=lambda i: (-order[i], i))[:k]
    return ranked + [-1] * (k - len(ranked))


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_score="max", renormalize=False, scale=1.0):
    """(weights [T, k] float64, experts [T, k])"""
    rows = logits.double().tolist()
    b = None if bias is None else bias.double().tolist()
    experts = [choose(l, k, score, b, groups, top_groups, group_score) for l in rows]
    weights = []
    for l, chosen in zip(rows, experts):
        if renormalize:                                       # of the chosen alone, so that small scores do not vanish
            x = [l[e] for e in chosen if e >= 0]
            top = max(x, default=0.0)
            raw = {e: math.exp(l[e] - top) * (1 if score == "softmax" else (1 + math.exp(top)) / (1 + math.exp(l[e])) if top < 700 else 1)
                   for e in chosen if e >= 0}
            total = sum(raw.values())
            weights.append([scale * raw[e] / total if e >= 0 else 0.0 for e in chosen])
        else:
            s = scores(l, score)
            weights.append([scale * s[e] if e >= 0 else 0.0 for e in chosen])
    return torch.tensor(weights, dtype=torch.float64).view(len(rows), k), torch.tensor(experts, dtype=torch.int32).view(len(rows), k)


def route_room(logits, k):
    """Relative error of a weight: the differences l - top lose half a step each of
    at most their span, expf and the division two steps each, the sums at most 16 + 6 + 6
    roundings (16 in a lane, then over 64 lanes); numerator and denominator both."""
    l = torch.where(torch.isfinite(logits.double()), logits.double(), torch.tensor(0.0, dtype=torch.float64))
    span = l.abs().amax(-1, keepdim=True) * 2 if l.numel() else l[:, :1]
    return (2 * span + 48) * U32


def route_grad(grad, logits, weights, experts, score, renormalize, scale):
    """(grad_logits [T, E] float64, the sum of the magnitudes that were added to each)"""
    T, E = logits.shape
    out, size = torch.zeros((T, E), dtype=torch.float64), torch.zeros((T, E), dtype=torch.float64)
    for t in range(T):
        l = logits[t].double().tolist()
        s = scores(l, score)
        pairs = [(e, float(grad[t, j]), float(weights[t, j])) for j, e in enumerate(experts[t].tolist()) if e >= 0]
        D, Da = sum(g * w for _, g, w in pairs), sum(abs(g * w) for _, g, w in pairs)
        for e, g, w in pairs:
            f = 1.0 if score == "softmax" else 1 - s[e] if s[e] < 0.5 else 1 / (1 + math.exp(l[e]))
            out[t, e] += w * f * (g - (D / scale if renormalize else 0.0))
            size[t, e] += w * f * (abs(g) + (Da / scale if renormalize else 0.0))
        if score == "softmax" and not renormalize:
            for e in range(E):
                if s[e] is not None:
                    out[t, e] -= s[e] * D
                    size[t, e] += s[e] * Da
    return out, size


def plan(experts, E):
    """(offsets, tokens, slots) by walking over the experts."""
    flat, k = experts.flatten().tolist(), experts.shape[1]
    offsets, tokens, slots = [0], [], [-1] * len(flat)
    for e in range(E):
        for p, x in enumerate(flat):
            if x == e:
                slots[p] = len(tokens)
                tokens.append(p // k)
        offsets.append(len(tokens))
    tokens += [-1] * (len(flat) - len(tokens))
    i32 = dict(dtype=torch.int32)
    return torch.tensor(offsets, **i32), torch.tensor(tokens, **i32), torch.tensor(slots, **i32).view(experts.shape)


def random_experts(seed, T, E, k, empty=0):
    """Distinct experts of each token; the last `empty` tokens have none."""
    g = torch.Generator().manual_seed(seed)
    e = torch.rand((T, E), generator=g).argsort(-1)[:, :k].int()
    e[T - empty:] = -1
    return e


def within(got, want, bound, what=""):
    g = got.detach().double().cpu()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    over = (g - want).abs() - bound
    assert not torch.isnan(g).any(), f"{what}: NaN"
    assert g.numel() == 0 or float(over.max()) <= 0, f"{what}: off by {float((g - want).abs().max()):.3e}, {float(over.max()):.3e} too far"


def rounded(bound, want, dtype):
    """The bound of a value known up to `bound` after its rounding to dtype."""
    return bound + U[dtype] * (want.abs() + bound) + 1e-38


def quantize(x):
    """x [M, K] -> (integers int64 [M, K], scale float32 [M]) from the definition."""
    x = x.double().numpy()
    top = np.abs(x).max(-1, initial=0.0)
    q, scale = np.zeros(x.shape, np.int64), np.zeros(x.shape[0], np.float32)
    for m in range(x.shape[0]):
        if not np.isfinite(top[m]):
            scale[m] = np.nan
        elif top[m] >= 2.0 ** -119:
            q[m] = np.rint(127.0 * x[m] / top[m]).astype(np.int64)
            scale[m] = np.float32(top[m]) / np.float32(127)
    return torch.from_numpy(q), torch.from_numpy(scale)


def product(q, s, w, sw, bias=None):
    """(y float64 of exact sums, bound of the fp32 steps: the sum's rounding, two products, the bias)."""
    y = (q.double() @ w.double().T) * sw.double() * s.double()[:, None]      # (integers below 2^53: exact)
    size = y.abs()
    if bias is not None:
        y, size = y + bias.double(), size + bias.double().abs()
    return y, 4.5 * U32 * size
