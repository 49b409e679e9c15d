"""Cases of the expert operators that stand around the grouped projections, and
of products in 8-bit integers.

A case is one pass through one operator:

  op "route"          a router's choice: scores of the logits, top-k of them
                      (with a bias for balance, in groups), the weights, and the
                      order in which the experts' products take the rows
  op "route-train"    the same, and the gradient of the logits
  op "gather"         each token's row to the places of its experts
  op "gather-train"   the same, and the gradient of the tokens' rows
  op "combine"        the experts' rows back to their tokens, weighted and summed
  op "combine-train"  the same, and the gradients of the rows and the weights
  op "int8"           a linear layer whose weight is held in 8-bit integers with a
                      scale for each channel; each token is quantised on the way
  op "int8-experts"   the same for a stack of experts, each token's row read from
                      where it stands

Where `own` is false the passes run in elementary torch operations in 32 bits
(64 for the order of scores, and 8-bit values are found without a rounding
before them); where it is true they are the calls a user makes.
"""

import math

import torch

own = False

PAD = 128          # a row of 8-bit integers is kept in a multiple of so many bytes
F32, BF16 = "float32", "bfloat16"


# ---- the cases ---------------------------------------------------------------
# 64 experts with 8 of them per token, 2048 wide, 1024 between, are the expert
# layers of this repository's benchmark; 4096/14336 and 5120/27648 its dense ones.

def listed():
    return [
        # one user, one new token: the whole call is latency
        dict(name="route-token", op="route", tokens=1, experts=64, k=8, score="softmax", bias=False, groups=1,
             top_groups=1, group_score="max", renormalize=False, scale=1.0, dtype=F32, padding=0),
        # a long prompt through a large balanced layer: groups are chosen first, then experts inside them
        dict(name="route-prompt", op="route", tokens=8191, experts=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renormalize=True, scale=2.5, dtype=F32, padding=0),
        # a fine-tuning step of packed samples with padding behind them
        dict(name="route-train", op="route-train", tokens=16384, experts=64, k=8, score="softmax", bias=False, groups=1,
             top_groups=1, group_score="max", renormalize=True, scale=1.0, dtype=BF16, padding=300),
        # one new token of each of 48 conversations
        dict(name="gather-batch", op="gather", tokens=48, experts=64, k=8, hidden=2048, dtype=BF16, padding=0, mix=1),
        # a fine-tuning step's tokens, some of them padding
        dict(name="gather-train", op="gather-train", tokens=4096, experts=64, k=8, hidden=2048, dtype=BF16, padding=77, mix=2),
        # 64 conversations in a wider model
        dict(name="combine-batch", op="combine", tokens=64, experts=128, k=8, hidden=5120, dtype=BF16, padding=0, mix=3),
        # a fine-tuning step's way back to the tokens
        dict(name="combine-train", op="combine-train", tokens=4095, experts=64, k=8, hidden=2048, dtype=BF16, padding=0, mix=4),
        # one user's next token through an attention projection
        dict(name="int8-token", op="int8", m=1, n=4096, inner=4096, dtype=BF16, out=BF16, bias=False),
        # a serving batch through an up projection
        dict(name="int8-batch", op="int8", m=32, n=14336, inner=4096, dtype=BF16, out=BF16, bias=False),
        # a prompt through an up projection of the largest layer
        dict(name="int8-prompt", op="int8", m=2048, n=27648, inner=5120, dtype=BF16, out=BF16, bias=False),
        # three conversations' next tokens through a stack of experts: a row or two each
        dict(name="int8-experts-token", op="int8-experts", tokens=3, experts=64, k=8, n=1024, inner=2048, dtype=BF16,
             out=BF16, padding=0, mix=5),
        # a prompt of 512 tokens through the same stack
        dict(name="int8-experts-prompt", op="int8-experts", tokens=512, experts=64, k=8, n=1024, inner=2048, dtype=BF16,
             out=BF16, padding=0, mix=6),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    if "padding" in case:
        case["padding"] = min(case["padding"], case["tokens"] // 2)
    return case


def _draw(rng):
    op = rng.choice(["route", "route", "route-train", "gather", "gather-train", "combine", "combine-train", "int8", "int8", "int8",
                     "int8-experts", "int8-experts"])
    dtype = rng.choice([BF16, BF16, F32])
    if op == "int8":
        inner = rng.choice([_log(rng, 40, 14336), 64 * _log(rng, 1, 224)])
        n = rng.choice([_log(rng, 24, 16384), 64 * _log(rng, 1, 256)])
        return dict(op=op, m=_log(rng, 1, min(8192, int(2.8e11 / (n * inner)))), n=n, inner=inner, dtype=dtype,
                    out=rng.choice([BF16, BF16, F32]), bias=rng.random() < 0.4)
    experts, k = rng.choice([(64, 8), (8, 2), (128, 8), (256, 8), (60, 4), (160, 6), (37, 1), (16, 4)])
    if op == "int8-experts":
        inner = rng.choice([_log(rng, 64, 4096), 64 * _log(rng, 1, 64)])
        n = rng.choice([1, 8]) * _log(rng, 8, max(8, min(512, int(1.3e8 / (experts * inner * 8)))))
        return dict(op=op, tokens=_log(rng, 1, 1024), experts=experts, k=k, n=n, inner=inner, dtype=dtype,
                    out=rng.choice([BF16, BF16, F32]), padding=rng.choice([0, 0, 3]), mix=rng.randrange(1 << 20))
    if op in ("route", "route-train"):
        groups = rng.choice([g for g in (1, 1, 4, 8) if experts % g == 0])
        top_groups = groups if groups == 1 else rng.choice([g for g in (1, 2, 3, 4) if g <= groups and g * (experts // groups) >= k])
        return dict(op=op, tokens=_log(rng, 1, 16384 * 64 // max(64, experts)), experts=experts, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, group_score=rng.choice(["max", "top2"]),
                    renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 1.0, 2.5]), dtype=dtype, padding=rng.choice([0, 0, 1, 25]))
    hidden = rng.choice([_log(rng, 64, 8192), 64 * _log(rng, 1, 128)])
    room = int(6.7e7 / (k * hidden * (2 if dtype == F32 else 1)))
    return dict(op=op, tokens=_log(rng, 1, max(1, min(16384, room))), experts=experts, k=k, hidden=hidden, dtype=dtype,
                padding=rng.choice([0, 0, 5]), mix=rng.randrange(1 << 20))


def experts_of(case):
    """The chosen experts int32 [tokens, k] on the host, from the case alone: some
    experts are asked for more than others; the last `padding` tokens have none (-1)."""
    g = torch.Generator()
    g.manual_seed(case["mix"])
    liking = 0.5 * torch.randn(case["experts"], generator=g)
    chosen = (torch.randn((case["tokens"], case["experts"]), generator=g) + liking).topk(case["k"], -1).indices.int()
    chosen[max(0, case["tokens"] - case["padding"]):] = -1
    return chosen


def work(case):
    op = case["op"]
    size = 2 if case["dtype"] == BF16 else 4
    if op == "int8":
        m, n, k = case["m"], case["n"], case["inner"]
        out = 2 if case["out"] == BF16 else 4
        return {"bytes": m * k * size + n * k + 4 * n + m * n * out, "flops": 2 * m * n * k}
    tokens, k = case["tokens"], case["k"]
    if op == "int8-experts":
        chosen = experts_of(case)
        rows, used = int((chosen >= 0).sum()), int(chosen[chosen >= 0].unique().numel())
        n, inner = case["n"], case["inner"]
        out = 2 if case["out"] == BF16 else 4
        return {"bytes": tokens * inner * size + used * n * (inner + 4) + tokens * k * (4 + n * out), "flops": 2 * rows * n * inner}
    if op in ("route", "route-train"):
        moved = tokens * case["experts"] * size + tokens * k * 4 * 4 + 4 * case["experts"]
        steps = 4 * tokens * case["experts"]
        if op == "route-train":
            moved, steps = moved + 2 * tokens * case["experts"] * size + 3 * 4 * tokens * k, 2 * steps
        return {"bytes": moved, "flops": steps}
    row, plan = case["hidden"] * size, 4 * tokens * k
    if op == "gather":
        return {"bytes": tokens * (1 + k) * row + plan, "flops": 0}
    if op == "gather-train":
        return {"bytes": 2 * (tokens * (1 + k) * row + plan), "flops": tokens * k * case["hidden"]}
    if op == "combine":
        return {"bytes": tokens * (1 + k) * row + 2 * plan, "flops": 2 * tokens * k * case["hidden"]}
    return {"bytes": tokens * (2 + 3 * k) * row + 5 * plan, "flops": 5 * tokens * k * case["hidden"]}


# ---- inputs --------------------------------------------------------------------

def _plan(chosen, experts):
    """chosen [T, k] (-1: none) -> offsets [experts + 1], the token of each row and
    the row of each choice (-1: none), rows sorted by expert, then by token."""
    flat = chosen.flatten().long()
    key = torch.where(flat < 0, experts, flat)
    order = torch.sort(key, stable=True).indices
    held = torch.zeros(experts + 1, dtype=torch.long, device=flat.device).index_add_(0, key, torch.ones_like(key))[:experts]
    offsets = torch.cat((held.new_zeros(1), held.cumsum(0)))
    there = torch.arange(flat.numel(), device=flat.device) < offsets[-1]
    tokens = torch.where(there, order // chosen.shape[1], -1)
    slots = torch.empty_like(order)
    slots[order] = torch.where(there, torch.arange(flat.numel(), device=flat.device), -1)
    return offsets.int(), tokens.int(), slots.view(chosen.shape).int()


def _integers(x):
    """x [rows, n] -> the integers -127 .. 127 nearest to 127 x / max |x| of the row
    (half-way to even) and the scale max / 127 of each row."""
    top = x.float().abs().amax(-1, keepdim=True)
    live = top >= 2.0 ** -119                                 # smaller rows are kept as zeros
    q = torch.round(127.0 * x.double() / torch.where(live, top, 1.0).double())
    return torch.where(live, q, 0.0).float(), torch.where(live, top / 127.0, 0.0)[:, 0]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    dtype, op = getattr(torch, case["dtype"]), case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    state = {"case": dict(case)}
    if op in ("route", "route-train"):
        tokens, experts = case["tokens"], case["experts"]
        logits = 1.5 * normal(tokens, experts) + 0.5 * normal(experts)
        logits[max(0, tokens - case["padding"]):] = -math.inf   # a padding token asks for nobody
        state["logits"] = logits.to(dtype)
        # what the balance rule has moved each expert by so far
        state["bias"] = 0.05 * normal(experts) if case["bias"] else None
        if op == "route-train":
            state["grad"] = normal(tokens, case["k"])
        return state
    if op in ("int8", "int8-experts"):
        inner, n = case["inner"], case["n"] * case.get("experts", 1)
        rows = case["m"] if op == "int8" else case["tokens"]
        # activations have a few strong channels
        state["x"] = (normal(rows, inner) * torch.exp(0.7 * normal(inner))).to(dtype)
        q, state["scale"] = torch.empty((n, -(-inner // PAD) * PAD), dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
        for at in range(0, n, 8192):
            part, state["scale"][at:at + 8192] = _integers(0.02 * normal(min(8192, n - at), inner))
            q[at:at + 8192] = torch.nn.functional.pad(part, (0, q.shape[1] - inner)).to(torch.int8)
        state["q"] = q
        if op == "int8":
            state["bias"] = normal(n) if case["bias"] else None
            return state
    state["experts"] = experts_of(case).to("cuda")
    state["offsets"], state["tokens"], state["slots"] = _plan(state["experts"], case["experts"])
    if op == "int8-experts":
        return state
    tokens, hidden, k = case["tokens"], case["hidden"], case["k"]
    if op.startswith("gather"):
        state["x"] = normal(tokens, hidden).to(dtype)
    else:
        state["y"] = normal(tokens * k, hidden).to(dtype)
    w = torch.exp(normal(tokens, k))
    state["weights"] = torch.where(state["experts"] >= 0, w / w.sum(-1, keepdim=True), 0.0)
    if op == "gather-train":
        state["grad"] = normal(tokens * k, hidden).to(dtype)
    elif op == "combine-train":
        state["grad"] = normal(tokens, hidden).to(dtype)
    return state


# ---- the plain form --------------------------------------------------------------

def _choose(case, logits, bias):
    """The experts of each token, in 64 bits: best first, equal ones by index, -1
    where no expert is left."""
    l = logits.double()
    live = l > -math.inf
    if case["score"] == "softmax":
        top = l.amax(-1, keepdim=True)
        e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        total = e.sum(-1, keepdim=True)
        s = e / torch.where(total > 0, total, 1.0)
    else:
        s = 1 / (1 + torch.exp(-l))
    c = s if bias is None else s + bias.double()
    c = torch.where(live, c, -math.inf)
    order = torch.where(live, l, -math.inf) if bias is None else c
    if case["groups"] > 1:
        g = c.view(c.shape[0], case["groups"], -1)
        if case["group_score"] == "max":
            of = (l if bias is None else c).view_as(g).amax(-1)
        else:
            two = g.sort(dim=-1, descending=True).values[..., :2]
            of = torch.where(two > -math.inf, two, 0.0).sum(-1)
            of = torch.where(two[..., 0] > -math.inf, of, -math.inf)
        first = of.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros_like(of, dtype=torch.bool).scatter_(1, first, True)
        order = torch.where(keep.repeat_interleave(g.shape[-1], 1), order, -math.inf)
    best = order.sort(dim=-1, descending=True, stable=True)
    return torch.where(best.values[:, :case["k"]] > -math.inf, best.indices[:, :case["k"]], -1)


def _plain_route(state, train):
    case, k = state["case"], state["case"]["k"]
    l = state["logits"].float()
    chosen = _choose(case, state["logits"], state["bias"])
    there, at = chosen >= 0, chosen.clamp(min=0)
    top = l.amax(-1, keepdim=True)
    if case["score"] == "softmax":
        e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        total = e.sum(-1, keepdim=True)
        s = e / torch.where(total > 0, total, 1.0)
    else:
        s = 1 / (1 + torch.exp(-l))
    picked = torch.where(there, s.gather(1, at), 0.0)
    total = picked.sum(-1, keepdim=True) if case["renormalize"] else torch.ones_like(picked[:, :1])
    share = picked / torch.where(total > 0, total, 1.0)
    weights = case["scale"] * share
    offsets, tokens, slots = _plan(chosen, case["experts"])
    out = {"weights": weights, "experts": chosen.int(), "offsets": offsets, "tokens": tokens, "slots": slots}
    if not train:
        return out
    g = torch.where(there, state["grad"], 0.0) * case["scale"]
    if case["renormalize"]:
        g = (g - (g * share).sum(-1, keepdim=True)) / torch.where(total > 0, total, 1.0)
    gs = torch.zeros_like(s).scatter_add_(1, at, torch.where(there, g, 0.0))
    if case["score"] == "softmax":
        gl = s * (gs - (gs * s).sum(-1, keepdim=True))
    else:
        gl = gs * s * (1 - s)
    out["grad_logits"] = gl.to(state["logits"].dtype)
    return out


def _rows_of(slots):
    return slots.flatten() >= 0, slots.flatten().clamp(min=0).long()


def _plain_gather(state, train):
    x, slots = state["x"], state["slots"]
    there, at = _rows_of(slots)
    tokens = state["tokens"]
    rows = x[tokens.clamp(min=0).long()] * (tokens >= 0)[:, None]
    if not train:
        return rows
    back = state["grad"].float()[at] * there[:, None]
    return {"rows": rows, "grad_x": back.view(*slots.shape, -1).sum(1).to(x.dtype)}


def _plain_combine(state, train):
    y, w, slots = state["y"], state["weights"], state["slots"]
    there, at = _rows_of(slots)
    each = (y.float()[at] * there[:, None]).view(*slots.shape, -1)
    out = (each * w[..., None]).sum(1).to(y.dtype)
    if not train:
        return out
    g = state["grad"].float()
    tokens = state["tokens"]
    weight = torch.zeros(slots.numel() + 1, device=w.device)
    weight[torch.where(there, at, slots.numel())] = w.flatten()
    gy = g[tokens.clamp(min=0).long()] * torch.where(tokens >= 0, weight[:-1], 0.0)[:, None]
    return {"out": out, "grad_y": gy.to(y.dtype), "grad_weights": (each * g[:, None]).sum(-1)}


def _plain_int8(state):
    case, inner = state["case"], state["case"]["inner"]
    q, scale = _integers(state["x"])
    y = torch.matmul(q, state["q"][:, :inner].float().T) * state["scale"] * scale[:, None]
    if state["bias"] is not None:
        y = y + state["bias"]
    return y.to(getattr(torch, case["out"]))


def _plain_int8_experts(state):
    case, inner, n = state["case"], state["case"]["inner"], state["case"]["n"]
    q, scale = _integers(state["x"])
    y = torch.zeros((state["tokens"].numel(), n), device=q.device)
    tokens = state["tokens"].clamp(min=0).long()
    ends = state["offsets"].tolist()
    for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        if a < b:
            rows = tokens[a:b]
            w = state["q"][e * n:(e + 1) * n, :inner].float()
            y[a:b] = torch.matmul(q[rows], w.T) * state["scale"][e * n:(e + 1) * n] * scale[rows][:, None]
    return y.to(getattr(torch, case["out"]))


# ---- one pass --------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "int8":
        return _plain_int8(state)
    if op == "int8-experts":
        return _plain_int8_experts(state)
    name, _, train = op.partition("-")
    return {"route": _plain_route, "gather": _plain_gather, "combine": _plain_combine}[name](state, train != "")


def _own(state, op):
    import nf4_bit_weight_amd as nf4

    case = state["case"]
    if op == "int8":
        w = nf4.NF4Int8(state["q"], state["scale"], case["n"], case["inner"])
        return nf4.nf4_int8_matmul(state["x"], w, bias=state["bias"], out_dtype=getattr(torch, case["out"]))
    if op == "int8-experts":
        w = nf4.NF4Int8(state["q"], state["scale"], case["n"], case["inner"])
        return nf4.nf4_int8_grouped_matmul(state["x"], state["offsets"], w, case["experts"], tokens=state["tokens"],
                                           out_dtype=getattr(torch, case["out"]))
    if op in ("route", "route-train"):
        how = dict(score=case["score"], bias=state["bias"], groups=case["groups"], top_groups=case["top_groups"],
                   group_score=case["group_score"], renormalize=case["renormalize"], scale=case["scale"])
        logits = state["logits"] if op == "route" else state["logits"].detach().requires_grad_()
        r = nf4.nf4_route(logits, case["k"], **how)
        out = {"weights": r.weights.detach(), "experts": r.experts, "offsets": r.offsets, "tokens": r.tokens, "slots": r.slots}
        if op == "route-train":
            out["grad_logits"], = torch.autograd.grad(r.weights, logits, state["grad"])
        return out
    r = nf4.NF4Routing(state["weights"], state["experts"], state["offsets"], state["tokens"], state["slots"])
    if op == "gather":
        return nf4.nf4_expert_gather(state["x"], r)
    if op == "combine":
        return nf4.nf4_expert_combine(state["y"], r)
    if op == "gather-train":
        x = state["x"].detach().requires_grad_()
        rows = nf4.nf4_expert_gather(x, r)
        gx, = torch.autograd.grad(rows, x, state["grad"])
        return {"rows": rows.detach(), "grad_x": gx}
    y = state["y"].detach().requires_grad_()
    r.weights = state["weights"].detach().requires_grad_()
    out = nf4.nf4_expert_combine(y, r)
    gy, gw = torch.autograd.grad(out, (y, r.weights), state["grad"])
    return {"out": out.detach(), "grad_y": gy, "grad_weights": gw}


# ---- the definition in 64 bits -----------------------------------------------------

def _exact_route(case, state, train):
    l = state["logits"].double().cpu()
    k, experts = case["k"], case["experts"]
    size = experts // case["groups"]
    live = ~torch.isneginf(l)
    if case["score"] == "softmax":
        s = torch.exp(l - torch.logsumexp(l, -1, keepdim=True))
        s = torch.where(live, s, 0.0)
    else:
        s = torch.sigmoid(l)
    bias = state["bias"]
    rank = l if bias is None else s + bias.double().cpu()
    c = s if bias is None else rank
    # one expert after another: the best of those left, the first of equal ones
    left = live.clone()
    if case["groups"] > 1:
        cg, lg = c.unflatten(-1, (-1, size)), live.unflatten(-1, (-1, size))
        by = rank.unflatten(-1, (-1, size)).masked_fill(~lg, -math.inf)
        best = by.amax(-1)
        if case["group_score"] == "top2":
            best = cg.masked_fill(~lg, -math.inf).amax(-1)
            one = cg.masked_fill(~lg, -math.inf).argmax(-1, keepdim=True)
            rest = cg.masked_fill(~lg, -math.inf).scatter(-1, one, -math.inf).amax(-1)
            best = torch.where(torch.isinf(rest), best, best + rest)
        taken = torch.zeros_like(best, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            i = best.masked_fill(taken, -math.inf).argmax(-1, keepdim=True)
            taken.scatter_(1, i, True)
        left &= taken.repeat_interleave(size, -1)
    chosen = torch.full((l.shape[0], k), -1, dtype=torch.long)
    for j in range(k):
        values = rank.masked_fill(~left, -math.inf)
        i = values.argmax(-1)
        some = left.any(-1)
        chosen[some, j] = i[some]
        left[torch.arange(l.shape[0])[some], i[some]] = False
    there, at = chosen >= 0, chosen.clamp(min=0)
    leaf = l.masked_fill(~live, -1e6).requires_grad_()
    s = torch.softmax(leaf, -1) if case["score"] == "softmax" else torch.sigmoid(leaf)
    picked = s.gather(1, at) * there
    if case["renormalize"]:
        total = picked.sum(-1, keepdim=True)
        picked = picked / torch.where(total > 0, total, 1.0)
    weights = case["scale"] * picked
    out = {"weights": weights.detach(), "experts": chosen.int()}
    # rows sorted by expert, counted one expert at a time
    flat, row, offsets = chosen.flatten(), 0, [0]
    tokens, slots = torch.full((flat.numel(),), -1, dtype=torch.int32), torch.full((flat.numel(),), -1, dtype=torch.int32)
    for e in range(experts):
        mine = torch.nonzero(flat == e)[:, 0]
        tokens[row:row + mine.numel()] = (mine // k).int()
        slots[mine] = torch.arange(row, row + mine.numel(), dtype=torch.int32)
        row += mine.numel()
        offsets.append(row)
    out.update(offsets=torch.tensor(offsets, dtype=torch.int32), tokens=tokens, slots=slots.view(-1, k))
    if train:
        gl, = torch.autograd.grad(weights, leaf, state["grad"].double().cpu() * there)
        out["grad_logits"] = gl
    return out


def _exact_int8(x, q, scale):
    """x [m, inner] through the weight q [n, inner] with its scales."""
    b = x.double()
    top = b.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -119)
    held = torch.round(b * 127 / top) * (top / 127)
    return held @ (q.double() * scale.double()[:, None]).T


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route-train"):
        return _exact_route(case, state, op == "route-train")
    if op == "int8":
        parts = [_exact_int8(state["x"], state["q"][a:a + 4096, :case["inner"]], state["scale"][a:a + 4096])
                 for a in range(0, case["n"], 4096)]
        y = torch.cat(parts, -1)
        return y if state["bias"] is None else y + state["bias"].double()
    offsets = state["offsets"].tolist()
    if op == "int8-experts":
        n = case["n"]
        y = torch.zeros((state["tokens"].numel(), n), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            a, b = offsets[e], offsets[e + 1]
            if a < b:
                part = slice(e * n, (e + 1) * n)
                y[a:b] = _exact_int8(state["x"][state["tokens"][a:b].long()], state["q"][part, :case["inner"]], state["scale"][part])
        return y
    # one choice of every token after another
    slots, k, tokens = state["slots"].long(), case["k"], case["tokens"]
    if op.startswith("gather"):
        rows = torch.zeros((tokens * k, case["hidden"]), dtype=torch.float64, device="cuda")
        gx = torch.zeros((tokens, case["hidden"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            has = slots[:, j] >= 0
            rows[slots[has, j]] = state["x"][has].double()
            if op == "gather-train":
                gx[has] += state["grad"][slots[has, j]].double()
        return rows if op == "gather" else {"rows": rows, "grad_x": gx}
    out = torch.zeros((tokens, case["hidden"]), dtype=torch.float64, device="cuda")
    gy = torch.zeros((tokens * k, case["hidden"]), dtype=torch.float64, device="cuda")
    gw = torch.zeros((tokens, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        has = slots[:, j] >= 0
        y, w = state["y"][slots[has, j]].double(), state["weights"][has, j].double()[:, None]
        out[has] += w * y
        if op == "combine-train":
            g = state["grad"][has].double()
            gy[slots[has, j]] = w * g
            gw[has, j] = (g * y).sum(-1)
    return out if op == "combine" else {"out": out, "grad_y": gy, "grad_weights": gw}
