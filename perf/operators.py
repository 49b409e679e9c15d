"""Cases of the attention operators that stand around the NF4 linear layers: a
paged key/value cache held in 4 bits (appending with the position rotation,
reading back, attention over it) and causal attention over packed prompts with
its backward pass.

A case is one pass through one operator:

  op "append"  rotate new queries and keys by their positions, quantise the
               keys and values into the cache's pages, and read the written
               rows back as the values the cache now stands for
  op "cache"   attention of the newest tokens of each sequence over its cache
  op "prompt"  causal attention over packed sequences, forward
  op "train"   the same, forward and backward

Where `own` is false the passes run in elementary torch operations in 32 bits
(64 for the rotation); where it is true they are the calls a user makes.
"""

import math
import random

import torch

own = False

# The sixteen values a stored 4-bit pattern stands for (sign, two exponent
# bits, one mantissa bit); a block of 64 shares one fp32 scale.
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 64
ROPE_BASE = 500000.0


# ---- the cases ---------------------------------------------------------------
# Head layouts: 32 query heads on 8 key heads of 128 (the 4096/1024-wide
# projections), 40 on 8 (5120/1024), 16 on 16 (2048-wide), and small ones of 64.

def listed():
    return [
        # one user, one new token: every launch is pure latency
        dict(name="append-token", op="append", batch=1, new=1, longest=4096, spread="same", mix=1,
             hq=32, hkv=8, dim=128, page=16, rotary=128, interleaved=False, keys=False),
        # a serving batch adds one token to each of 64 conversations
        dict(name="append-batch", op="append", batch=64, new=1, longest=8192, spread="even", mix=2,
             hq=40, hkv=8, dim=128, page=64, rotary=128, interleaved=False, keys=False),
        # nine prompts of different lengths enter the cache at once; the rotated keys go on to the prompt's attention
        dict(name="append-prompts", op="append", batch=9, new=0, longest=3001, spread="even", mix=3,
             hq=32, hkv=8, dim=128, page=64, rotary=128, interleaved=False, keys=True),
        # the start of one conversation: a few hundred keys, no grouping of heads
        dict(name="cache-short", op="cache", batch=1, new=1, longest=257, spread="same", mix=4,
             hq=16, hkv=16, dim=128, page=16),
        # one very long document: all of the machine has to work on one sequence
        dict(name="cache-long", op="cache", batch=1, new=1, longest=131071, spread="same", mix=5,
             hq=32, hkv=8, dim=128, page=64),
        # a serving batch in full swing, lengths from one token to 8192
        dict(name="cache-batch", op="cache", batch=64, new=1, longest=8192, spread="even", mix=6,
             hq=32, hkv=8, dim=128, page=64),
        # five guessed tokens of each sequence are checked at once; pages that no tile divides
        dict(name="cache-verify", op="cache", batch=16, new=5, longest=4099, spread="even", mix=7,
             hq=40, hkv=8, dim=128, page=48),
        # a chat turn of one user
        dict(name="prompt-short", op="prompt", batch=1, longest=77, spread="same", mix=8, hq=32, hkv=8, dim=128),
        # a long document read at once
        dict(name="prompt-long", op="prompt", batch=1, longest=8192, spread="same", mix=9, hq=32, hkv=8, dim=128),
        # a batch of prompts of uneven lengths, packed
        dict(name="prompt-packed", op="prompt", batch=12, longest=2049, spread="even", mix=10, hq=40, hkv=8, dim=128),
        # a fine-tuning step on packed samples
        dict(name="train-packed", op="train", batch=6, longest=2048, spread="even", mix=11, hq=32, hkv=8, dim=128),
        # fine-tuning a small model on short samples
        dict(name="train-small", op="train", batch=5, longest=203, spread="log", mix=12, hq=8, hkv=2, dim=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv, dim = rng.choice([(32, 8, 128), (40, 8, 128), (16, 16, 128), (8, 2, 64), (12, 4, 64), (7, 1, 128), (64, 8, 64)])
    case = dict(op=rng.choice(["append", "cache", "prompt", "train"]), spread=rng.choice(["same", "even", "log"]),
                mix=rng.randrange(1 << 20), hq=hq, hkv=hkv, dim=dim)
    if case["op"] in ("append", "cache"):
        case.update(page=rng.choice([16, 32, 48, 64, 128, 256]))
    if case["op"] == "append":
        batch = _log(rng, 1, 64)
        case.update(batch=batch, new=rng.choice([0, 1, 1, 3]), longest=_log(rng, 3, max(3, 15000 // batch)),
                    rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3, keys=rng.random() < 0.5)
    elif case["op"] == "cache":
        batch = _log(rng, 1, 64)
        case.update(batch=batch, new=rng.choice([1, 1, 2, 4, 5, 9]), longest=_log(rng, 1, min(262144, (1 << 28) // (hkv * dim * batch))))
    else:
        batch = _log(rng, 1, 16)
        case.update(batch=batch, longest=_log(rng, 1, int((1.2e7 / batch) ** 0.5)))
    return case


def lengths_of(case):
    """The sequences' lengths, from the case alone: all the longest ("same"),
    evenly spread from one up, or spread over their logarithm."""
    r, b, top = random.Random(case["mix"]), case["batch"], case["longest"]
    if case["spread"] == "same":
        got = [top] * b
    elif case["spread"] == "even":
        got = [r.randint(1, top) for _ in range(b)]
    else:
        got = [_log(r, 1, top) for _ in range(b)]
    got[r.randrange(b)] = top
    return got


def new_of(case):
    """New tokens per sequence (0 in the case: the whole sequence is new)."""
    lens = lengths_of(case)
    return [n if case["new"] == 0 else min(n, case["new"]) for n in lens]


def work(case):
    d, hq, hkv, lens = case["dim"], case["hq"], case["hkv"], lengths_of(case)
    if case["op"] in ("append", "cache"):
        new = new_of(case)
        rows = sum(new)
        held = hkv * (d // 2 + d // BLOCK * 4)              # bytes of one token's keys (or values) in the cache
        if case["op"] == "append":
            # q in and out, k and v in, codes and scales out and in again, the values out
            moved = rows * (4 * hq * d + 4 * hkv * d + 4 * held + 4 * hkv * d + (2 * hkv * d if case["keys"] else 0))
            return {"bytes": moved, "flops": rows * (hq + 2 * hkv) * d * 4}
        pairs = sum(n * ln - n * (n - 1) // 2 for n, ln in zip(new, lens))
        return {"bytes": 2 * held * sum(lens) + 4 * rows * hq * d, "flops": 4 * hq * d * pairs}
    rows, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
    if case["op"] == "prompt":
        return {"bytes": 2 * rows * d * (2 * hq + 2 * hkv), "flops": 4 * hq * d * pairs}
    # forward two products; backward five (scores again, dP, dV, dK, dQ)
    return {"bytes": 2 * rows * d * (4 * hq + 4 * hkv), "flops": (4 + 10) * hq * d * pairs}


# ---- inputs --------------------------------------------------------------------

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _sums(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    d, hq, hkv, lens = case["dim"], case["hq"], case["hkv"], lengths_of(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    state = {"case": dict(case)}
    if case["op"] in ("prompt", "train"):
        rows = sum(lens)
        state["offsets"] = _i32(_sums(lens))
        state["q"] = normal(rows, hq, d).to(torch.bfloat16)
        state["k"] = normal(rows, hkv, d).to(torch.bfloat16)
        state["v"] = normal(rows, hkv, d).to(torch.bfloat16)
        if case["op"] == "train":
            state["gy"] = normal(rows, hq, d).to(torch.bfloat16)
        return state

    new, page = new_of(case), case["page"]
    rows = sum(new)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [0] * (max(need) - n))
        at += n
    state["page_table"] = _i32(table)
    state["lengths"] = _i32(lens)
    state["offsets"] = _i32(_sums(new))
    state["q"] = normal(rows, hq, d).to(torch.bfloat16)
    # keys have strong and weak channels
    channel = torch.exp(0.5 * normal(1, hkv, 1, d))
    if case["op"] == "append":
        state["k"] = (normal(rows, hkv, d) * channel[:, :, 0]).to(torch.bfloat16)
        state["v"] = normal(rows, hkv, d).to(torch.bfloat16)
        half = case["rotary"] // 2
        state["inv_freq"] = (ROPE_BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        for name in ("k", "v"):
            state[name + "_codes"] = torch.zeros((pages, hkv, page, d // 2), dtype=torch.uint8, device="cuda")
            state[name + "_scale"] = torch.zeros((pages, hkv, page, d // BLOCK), dtype=torch.float32, device="cuda")
    else:
        # what earlier calls left in the cache
        for name in ("k", "v"):
            x = normal(pages, hkv, page, d)
            x = (x * channel if name == "k" else x).to(torch.bfloat16)
            state[name + "_codes"], state[name + "_scale"] = _quantise(x)
            del x
    return state


# ---- the plain form --------------------------------------------------------------

def _quantise(x):
    """x [..., d] bf16 -> two 4-bit patterns a byte (the first in the high
    half) and the fp32 scale of each block of 64."""
    b = x.float().reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    live = top >= 2.0 ** -120                                  # smaller blocks are kept as zeros
    # |x| / (top / 6) against the middles between levels, half-way going outwards: with eighths of both
    # sides every product of these 8-bit numbers is exact
    m, t = 0.75 * b.abs(), 0.125 * top
    code = ((m >= 0.25 * t).byte() + (m >= 0.75 * t) + (m >= 1.25 * t) + (m >= 1.75 * t) + (m >= 2.5 * t) + (m >= 3.5 * t) + (m >= 5.0 * t))
    code = torch.where(live, code + 8 * torch.signbit(b).byte(), 0).byte()
    code = code.reshape(*x.shape[:-1], -1, 2)
    scale = torch.where(live, top / 6.0, torch.zeros_like(top))
    return (code[..., 0] * 16 + code[..., 1]).contiguous(), scale[..., 0].contiguous()


def _values(codes, scale):
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float32, device=codes.device)
    at = torch.stack((codes >> 4, codes & 15), -1).flatten(-2).int()
    return (levels[at].unflatten(-1, (-1, BLOCK)) * scale[..., None]).flatten(-2)


def _rotate(x, angle, half, interleaved):
    """The pairs of the first 2 * half elements turned by angle [rows, half], in 64 bits, rounded once."""
    y = x.double()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half])
    u, w = a * c - b * s, b * c + a * s
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., 2 * half:]), -1).float().to(torch.bfloat16)


def _places(state, rows):
    """Sequence, position, page and place in the page of each new row."""
    off, at = state["offsets"].long(), torch.arange(rows, device="cuda")
    seq = torch.searchsorted(off, at, right=True) - 1
    pos = state["lengths"].long()[seq] - off[seq + 1] + at
    page = state["case"]["page"]
    return pos, state["page_table"][seq, pos // page].long(), pos % page


def _plain_append(state):
    case, k, v = state["case"], state["k"], state["v"]
    pos, page, place = _places(state, k.shape[0])
    half = case["rotary"] // 2
    angle = pos.double()[:, None] * state["inv_freq"].double()[None]
    q = _rotate(state["q"], angle, half, case["interleaved"])
    k = _rotate(k, angle, half, case["interleaved"])
    state["k_codes"][page, :, place], state["k_scale"][page, :, place] = _quantise(k)
    state["v_codes"][page, :, place], state["v_scale"][page, :, place] = _quantise(v)
    held = (_values(state["k_codes"][page, :, place], state["k_scale"][page, :, place]).to(torch.bfloat16),
            _values(state["v_codes"][page, :, place], state["v_scale"][page, :, place]).to(torch.bfloat16))
    return {"q": q, "k": k if case["keys"] else None, "held_k": held[0], "held_v": held[1]}


def _padded(x, offsets, longest):
    """Packed rows [T, ...] -> [B, longest, ...] and the truth of each place."""
    at = torch.arange(longest, device=x.device)[None]
    off = offsets.long()
    there = at < (off[1:] - off[:-1])[:, None]
    return x[torch.where(there, off[:-1, None] + at, 0)], there


def _packed(y, there, rows):
    """[B, longest, ...] back to packed rows."""
    at = torch.where(there, torch.cumsum(there.flatten(), 0).view_as(there) - 1, rows)
    out = torch.zeros((rows + 1, *y.shape[2:]), dtype=y.dtype, device=y.device)
    out[at] = y
    return out[:rows]


def _softmax(s, seen):
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total)


def _plain_cache(state):
    case, q = state["case"], state["q"]
    hkv, d, page, group = case["hkv"], case["dim"], case["page"], case["hq"] // case["hkv"]
    n, batch = max(new_of(case)), case["batch"]
    table = state["page_table"].long()
    span = table.shape[1] * page

    def dense(name):                                          # [B, hkv, span, d]
        x = _values(state[name + "_codes"][table], state[name + "_scale"][table])
        return x.transpose(1, 2).reshape(batch, hkv, span, d)

    qp, there = _padded(q.float(), state["offsets"], n)        # [B, n, hq, d]
    qp = qp.view(batch, n, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, n * group, d)
    s = torch.matmul(qp, dense("k").transpose(-1, -2).contiguous()) / math.sqrt(d)
    off, at = state["offsets"].long(), torch.arange(n, device="cuda")
    pos = (state["lengths"].long() - (off[1:] - off[:-1]))[:, None] + at[None]                  # [B, n]
    seen = torch.arange(span, device="cuda")[None, None] <= pos[..., None]                      # [B, n, span]
    p = _softmax(s, seen[:, None, :, None].expand(-1, 1, -1, group, -1).reshape(batch, 1, n * group, span))
    o = torch.matmul(p, dense("v")).view(batch, hkv, n, group, d).permute(0, 2, 1, 3, 4).reshape(batch, n, hkv * group, d)
    return _packed(o, there, q.shape[0]).to(torch.bfloat16)


def _plain_prompt(state, train):
    case = state["case"]
    hkv, d, group, batch, n = case["hkv"], case["dim"], case["hq"] // case["hkv"], case["batch"], case["longest"]
    rows, off = state["q"].shape[0], state["offsets"]

    def heads(x):                                             # [B, hkv, group * n, d] of queries, [B, hkv, n, d] of keys
        x, there = _padded(x.float(), off, n)
        x = x * there[..., None, None]
        return x.view(batch, n, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d), there

    def rows_of(y, h):
        y = y.view(batch, hkv, h // hkv, n, d).permute(0, 3, 1, 2, 4).reshape(batch, n, h, d)
        return _packed(y, there, rows).to(torch.bfloat16)

    (q, there), (k, _), (v, _) = heads(state["q"]), heads(state["k"]), heads(state["v"])
    at = torch.arange(n, device="cuda")
    seen = at[None] <= at[:, None]
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()).view(batch, hkv, group, n, n) / math.sqrt(d)
    p = _softmax(s, seen).view(batch, hkv, group * n, n)
    del s
    out = rows_of(torch.matmul(p, v), hkv * group)
    if not train:
        return out
    gy, _ = heads(state["gy"])
    gv = torch.matmul(p.transpose(-1, -2).contiguous(), gy)
    gp = torch.matmul(gy, v.transpose(-1, -2).contiguous())
    gs = p * (gp - (p * gp).sum(-1, keepdim=True)) / math.sqrt(d)
    del gp, p
    gq = torch.matmul(gs, k)
    gk = torch.matmul(gs.transpose(-1, -2).contiguous(), q)
    return {"out": out, "grad_q": rows_of(gq, hkv * group), "grad_k": rows_of(gk, hkv), "grad_v": rows_of(gv, hkv)}


# ---- one pass --------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "append":
        return _plain_append(state)
    if op == "cache":
        return _plain_cache(state)
    return _plain_prompt(state, op == "train")


def _own(state, op):
    import nf4_bit_weight_amd as nf4

    case, off = state["case"], state["offsets"]
    if op == "prompt":
        return nf4.nf4_prompt_attention(state["q"], state["k"], state["v"], off)
    if op == "train":
        q, k, v = (state[n].detach().requires_grad_() for n in "qkv")
        out = nf4.nf4_prompt_attention(q, k, v, off)
        gq, gk, gv = torch.autograd.grad(out, (q, k, v), state["gy"])
        return {"out": out.detach(), "grad_q": gq, "grad_k": gk, "grad_v": gv}
    cache = nf4.NF4KVCache(state["k_codes"], state["k_scale"], state["v_codes"], state["v_scale"])
    lens, table = state["lengths"], state["page_table"]
    if case["new"] == 1:
        off = None                                             # one new token of every sequence
    if op == "cache":
        return nf4.nf4_kv_attention(state["q"], cache, lens, table, offsets=off)
    q, k = nf4.nf4_kv_append(cache, state["k"], state["v"], lens, table, offsets=off, inv_freq=state["inv_freq"],
                             interleaved=case["interleaved"], q=state["q"], return_k=case["keys"])
    held_k, held_v = nf4.nf4_kv_dequantize(cache, lens, table, offsets=off, rows=state["k"].shape[0])
    return {"q": q, "k": k, "held_k": held_k, "held_v": held_v}


# ---- the definition in 64 bits -----------------------------------------------------

def _exact_values(codes, scale):
    c = codes.long()
    out = torch.zeros((*c.shape[:-1], 2 * c.shape[-1]), dtype=torch.float64, device=c.device)
    for i, nib in ((0, c // 16), (1, c % 16)):
        e, m = (nib % 8) // 2, nib % 2
        mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e - 1).double())
        out[..., i::2] = torch.where(nib >= 8, -mag, mag)
    return out * scale.double().repeat_interleave(BLOCK, -1)


def _exact_round(x):
    """Nearest of the sixteen values, half-way going outwards."""
    e = torch.floor(torch.log2(x.abs().clamp(min=1.0))).clamp(max=2)
    step = 2.0 ** (e - 1)
    return torch.sign(x) * torch.floor(x.abs() / step + 0.5) * step


def _exact_append(case, state):
    rows, half = state["k"].shape[0], case["rotary"] // 2
    new, lens = new_of(case), lengths_of(case)
    pos = torch.cat([torch.arange(ln - n, ln) for n, ln in zip(new, lens)]).double()
    turn = torch.polar(torch.ones(rows, half, dtype=torch.float64), pos[:, None] * state["inv_freq"].cpu().double())[:, None]

    def rotated(x):
        x = x.cpu().double()
        first = x[..., :2 * half]
        if case["interleaved"]:
            z = torch.view_as_complex(first.unflatten(-1, (half, 2)).contiguous()) * turn
            first = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(first[..., :half], first[..., half:]) * turn
            first = torch.cat((z.real, z.imag), -1)
        return torch.cat((first, x[..., 2 * half:]), -1)

    def held(x):                                               # of the values the cache is given, in bf16
        b = x.float().to(torch.bfloat16).double().unflatten(-1, (-1, BLOCK))
        top = b.abs().amax(-1, keepdim=True)
        return (_exact_round(6 * b / top) * (top / 6)).flatten(-2)

    q, k = rotated(state["q"]), rotated(state["k"])
    return {"q": q, "k": k if case["keys"] else None, "held_k": held(k), "held_v": held(state["v"].cpu())}


def _exact_attend(q, k, v, pos, scale):
    """q [n, hq, d] at positions pos over k, v [L, hkv, d], all in 64 bits."""
    group = q.shape[1] // k.shape[1]
    out = torch.zeros_like(q)
    for h in range(q.shape[1]):
        s = (q[:, h] @ k[:, h // group].T) * scale
        s = s.masked_fill(torch.arange(k.shape[0], device=q.device)[None] > pos[:, None], -math.inf)
        out[:, h] = torch.softmax(s, -1) @ v[:, h // group]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, state)
    d, lens = case["dim"], lengths_of(case)
    scale = 1 / math.sqrt(d)
    if case["op"] == "cache":
        new, outs, at = new_of(case), [], 0
        for b, (n, ln) in enumerate(zip(new, lens)):
            pages = state["page_table"][b, :-(-ln // case["page"])].long()
            k, v = (_exact_values(state[x + "_codes"][pages], state[x + "_scale"][pages])
                    .transpose(1, 2).flatten(0, 1)[:ln] for x in "kv")
            outs.append(_exact_attend(state["q"][at:at + n].double(), k, v, torch.arange(ln - n, ln, device="cuda"), scale))
            at += n
        return torch.cat(outs)
    if sum(n * n for n in lens) * case["hq"] > 2.2e9:
        return None
    leaves = [state[x].double().requires_grad_(case["op"] == "train") for x in "qkv"]
    off = _sums(lens)
    outs = []
    for a, b in zip(off[:-1], off[1:]):
        q, k, v = (x[a:b] for x in leaves)
        group = case["hq"] // case["hkv"]
        k, v = (x.repeat_interleave(group, 1) for x in (k, v))
        s = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0)) * scale
        s = s + torch.full((b - a, b - a), -math.inf, dtype=torch.float64, device="cuda").triu(1)
        outs.append(torch.matmul(torch.softmax(s, -1), v.transpose(0, 1)).transpose(0, 1))
    out = torch.cat(outs)
    if case["op"] == "prompt":
        return out
    gq, gk, gv = torch.autograd.grad(out, leaves, state["gy"].double())
    return {"out": out.detach(), "grad_q": gq, "grad_k": gk, "grad_v": gv}
