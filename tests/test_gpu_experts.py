"""The expert operators against plain 64-bit forms: the choice and its plan are
compared whole, weights, rows and gradients to bounds counted from the
roundings."""

import itertools
import math

import pytest
import torch

import expert_ref as R
from nf4_bit_weight_amd import (NF4Routing, nf4_expert_combine, nf4_expert_combine_bwd, nf4_expert_gather,
                                nf4_expert_gather_bwd, nf4_expert_plan, nf4_route, nf4_route_bwd)
from nf4_bit_weight_amd._lib import NF4Error

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
INF = math.inf


def check_route(logits, k, **how):
    r = nf4_route(logits.to(DEV), k, **{n: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for n, v in how.items()})
    w, e = R.route(logits, k, **how)
    assert torch.equal(r.experts.cpu(), e), how
    R.within(r.weights, w, R.route_room(logits, k) * w + 1e-38, str(how))
    for got, want in zip((r.offsets, r.tokens, r.slots), R.plan(e, logits.shape[1])):
        assert torch.equal(got.cpu(), want)
    return r


# one to eight experts a token, every number of lanes a token, odd counts
SHAPES = [(1, 1, 1), (3, 2, 2), (65, 8, 8), (33, 9, 2), (70, 16, 5), (17, 31, 31), (130, 60, 4), (1, 64, 8), (129, 64, 8),
          (40, 100, 7), (19, 128, 1), (9, 200, 64), (23, 256, 8), (5, 511, 3), (6, 512, 10), (7, 513, 6), (3, 1024, 64)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", R.BOTH)
def test_route_shapes(T, E, k, dtype):
    l = (2 * R.normal(T * 7 + E, T, E)).to(dtype)
    check_route(l, k)
    check_route(l, k, score="sigmoid", renormalize=True, scale=2.5)
    check_route(l, k, score="sigmoid", bias=0.1 * R.normal(E, E))
    check_route(l, k, bias=0.02 * R.normal(E, E), renormalize=True)


@pytest.mark.parametrize("T,E,k,groups,top", [(37, 64, 8, 8, 4), (5, 256, 8, 8, 4), (11, 256, 6, 16, 3), (9, 60, 4, 4, 2), (4, 8, 2, 8, 2),
                                              (3, 16, 2, 2, 1), (2, 1024, 8, 64, 8), (6, 120, 3, 40, 5), (7, 33, 3, 11, 11),
                                              (2, 900, 20, 3, 2), (3, 64, 8, 64, 20)])
@pytest.mark.parametrize("rank", ["max", "top2"])
def test_route_groups(T, E, k, groups, top, rank):
    l = R.normal(E + groups, T, E)
    for score, bias in itertools.product(("softmax", "sigmoid"), (None, 0.05 * R.normal(3, E))):
        check_route(l, k, score=score, bias=bias, groups=groups, top_groups=top, group_score=rank, renormalize=True)


@pytest.mark.parametrize("E", [8, 64, 300])
def test_equal_scores_go_to_the_lower_index(E):
    l = torch.zeros(5, E)
    l[1] = torch.arange(E) % 3                                  # runs of equal logits
    l[2, E // 2:] = -0.0
    l[3] = torch.finfo(torch.float32).min
    l[4] = (torch.arange(E) // 2 % 2).float()
    for how in (dict(), dict(score="sigmoid", bias=torch.zeros(E)), dict(groups=4, top_groups=2),
                dict(groups=4, top_groups=2, group_score="top2", score="sigmoid")):
        if E % how.get("groups", 1) == 0:
            check_route(l, min(8, E), **how)


def test_close_scores_are_told_apart():
    """Sums of score and bias that fp32 does not tell apart keep the order of the numbers."""
    E = 64
    l = torch.zeros(E)
    bias = torch.zeros(E)
    l[5], bias[5] = 1.0, 0.0
    s = 1 / (1 + math.exp(-1.0))
    bias[9] = s - 0.5                                           # expert 9: 0.5 + fp32(s - 0.5)
    for i in range(10, 30):
        bias[i] = torch.nextafter(bias[9], torch.tensor(1.0 if i % 2 else 0.0)) if i < 20 else bias[9]
    check_route(l[None].expand(3, E), 30, score="sigmoid", bias=bias)


@pytest.mark.parametrize("E", [16, 64, 512])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(E, score):
    l = R.normal(E, 9, E)
    l[0] = -INF                                                 # nobody
    l[1, 1:] = -INF                                             # one
    l[2, ::2] = -INF
    l[3, : E // 4] = -INF                                       # a whole group
    l[4] = torch.finfo(torch.float32).min                       # the type's lowest value is a number
    l[5, 3] = torch.finfo(torch.float32).min
    l[6, 4:] = -INF
    l[7, [0, E // 4, E // 2]] = -INF
    l[8, 5:] = torch.finfo(torch.float32).min
    bias = 0.01 * R.normal(1, E)
    bias[7] = -INF                                              # an expert out of service
    for how in (dict(), dict(renormalize=True), dict(bias=bias, renormalize=True), dict(groups=4, top_groups=2, renormalize=True),
                dict(groups=4, top_groups=2, group_score="top2"), dict(groups=4, top_groups=2, group_score="top2", bias=bias)):
        check_route(l, 6, score=score, **how)
    b = l[:4].to(torch.bfloat16)
    b[2, 1] = torch.finfo(torch.bfloat16).min
    check_route(b, 6, score=score)


def test_far_logits_keep_their_weights():
    """Renormalised weights do not vanish with the scores that they are made of."""
    l = torch.full((4, 64), -200.0)
    l[0, :8] = torch.arange(8.0) - 150
    l[1, :3] = 300.0
    l[2] = -90.0 + R.normal(2, 64)
    l[3, 5] = 80.0
    for score in ("softmax", "sigmoid"):
        r = check_route(l, 8, score=score, renormalize=True)
        assert (r.weights.sum(-1) - 1).abs().max() < 1e-5


def test_nan_logits_are_seen():
    """A NaN reaches the weights of its own token only, and the choice stays in range."""
    l = R.normal(3, 4, 64)
    l[1, 17] = math.nan
    l[2, 5] = INF
    for how in (dict(), dict(score="sigmoid"), dict(bias=torch.zeros(64)), dict(groups=8, top_groups=2, group_score="top2")):
        how = {n: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for n, v in how.items()}
        r = nf4_route(l.to(DEV), 8, **how)
        assert torch.isnan(r.weights[1]).any()
        assert ((r.experts >= 0) & (r.experts < 64)).all()
        assert all(len(set(row)) == 8 for row in r.experts.tolist())
        if how.get("score") != "sigmoid":
            assert torch.isnan(r.weights[2]).any()
        assert torch.isfinite(r.weights[[0, 3]]).all()


def test_route_takes_strided_rows_and_other_types():
    joint = R.normal(4, 31, 100).to(DEV)
    for piece in (joint[:, 8:72], joint[:, 3:67], joint[::2, :64]):
        check_route(piece.cpu(), 8)
        r, want = nf4_route(piece, 8), nf4_route(piece.contiguous(), 8)
        assert torch.equal(r.weights, want.weights) and torch.equal(r.slots, want.slots)
    t = joint.t()[:64]                                          # [64, 31], columns apart: copied
    assert torch.equal(nf4_route(t, 4).experts, nf4_route(t.contiguous(), 4).experts)
    h = joint.half()
    assert torch.equal(nf4_route(h, 4).weights, nf4_route(h.float(), 4).weights)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (70, 64, 8), (33, 100, 5), (9, 256, 8), (4, 1000, 20)])
@pytest.mark.parametrize("dtype", R.BOTH)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient(T, E, k, dtype, score, renormalize):
    l = (1.5 * R.normal(T + E, T, E)).to(dtype)
    if T > 4:
        l[1] = -INF
        l[2, 2:] = -INF
        l[3, E // 2] = torch.finfo(dtype).min
    g = R.normal(5, T, k)
    how = dict(score=score, renormalize=renormalize, scale=1.75)
    leaf = l.to(DEV).requires_grad_()
    r = nf4_route(leaf, k, **how)
    got, = torch.autograd.grad(r.weights, leaf, g.to(DEV))
    assert got.dtype == dtype
    w = r.weights.detach().cpu()
    want, size = R.route_grad(g, l, w, r.experts.cpu(), score, renormalize, 1.75)
    R.within(got, want, R.rounded((R.route_room(l, k) + 2 * k * R.U32) * size, want, dtype), f"{how}")
    assert torch.equal(got, nf4_route_bwd(g.to(DEV), leaf.detach(), r, **how))


def test_route_gradient_against_differences():
    T, E, k, h = 6, 24, 4, 1e-5
    l = R.normal(8, T, E).double()
    g = R.normal(9, T, k)
    for score, renorm in itertools.product(("softmax", "sigmoid"), (False, True)):
        leaf = l.float().to(DEV).requires_grad_()
        r = nf4_route(leaf, k, score=score, renormalize=renorm)
        got, = torch.autograd.grad(r.weights, leaf, g.to(DEV))
        base = l.float().double()
        for t, e in itertools.product(range(T), range(0, E, 5)):
            two = []
            for d in (h, -h):
                x = base.clone()
                x[t, e] += d
                w, ex = R.route(x, k, score=score, renormalize=renorm)
                assert torch.equal(ex, r.experts.cpu())
                two.append(float((w * g.double()).sum()))
            # error of a central difference: h^2 / 6 times the third derivative (at most 8 sum |g|), and 64-bit rounding / h
            room = 8 * float(g.abs()[t].sum()) * h * h + 1e-9 + 60 * R.U32 * float(g.abs()[t].sum())
            assert abs(float(got[t, e]) - (two[0] - two[1]) / (2 * h)) <= room


@pytest.mark.parametrize("T,E,k,empty", [(0, 4, 2, 0), (1, 1, 1, 0), (1, 64, 8, 0), (7, 5, 3, 2), (128, 64, 8, 0), (129, 64, 8, 40),
                                         (300, 256, 8, 1), (1100, 37, 3, 0), (260, 600, 4, 0), (130, 1024, 2, 9), (50, 3, 1, 50)])
def test_plan(T, E, k, empty):
    e = R.random_experts(T + E, T, E, k, empty)
    for got, want in zip(nf4_expert_plan(e.to(DEV), E), R.plan(e, E)):
        assert torch.equal(got.cpu(), want)


def test_plan_of_any_integers():
    """The same expert named twice by a token, numbers that name nobody, more choices than experts."""
    g = torch.Generator().manual_seed(2)
    e = torch.randint(-3, 9, (500, 6), generator=g, dtype=torch.int32)
    e[3] = 2
    e[4, 0], e[5, 1] = 2 ** 31 - 1, -2 ** 31
    for got, want in zip(nf4_expert_plan(e.to(DEV), 5), R.plan(e, 5)):
        assert torch.equal(got.cpu(), want)
    same = torch.full((700, 8), 1, dtype=torch.int32)           # one expert takes all
    for got, want in zip(nf4_expert_plan(same.to(DEV), 3), R.plan(same, 3)):
        assert torch.equal(got.cpu(), want)


def sorted_plan(e, E):
    flat, k = e.flatten().long(), e.shape[1]
    flat = torch.where((flat < 0) | (flat >= E), E, flat)
    order, count = flat.argsort(stable=True), flat.bincount(minlength=E + 1)
    offsets, used = torch.cat([count.new_zeros(1), count[:E].cumsum(0)]), int(count[:E].sum())
    tokens, slots = torch.full_like(flat, -1), torch.full_like(flat, -1)
    tokens[:used] = order[:used] // k
    slots[order[:used]] = torch.arange(used)
    return offsets.int(), tokens.int(), slots.int().view(e.shape)


@pytest.mark.parametrize("T,E,k", [(9000, 2, 1), (9001, 8, 8), (5000, 11, 3), (3000, 32, 4), (1500, 64, 6), (1501, 120, 8), (700, 256, 8),
                                   (16390, 256, 2), (400, 500, 5), (330, 1000, 3), (5000, 1024, 4), (40000, 600, 1)])
def test_plan_of_many_runs(T, E, k):
    """Every width of the counts, from few workgroups' to those that are summed beforehand."""
    logits = R.normal(T + E, T, E)
    logits[::7] = -float("inf")
    r = nf4_route(logits.to(DEV), k)
    for got, want, plan in zip((r.offsets, r.tokens, r.slots), sorted_plan(r.experts.cpu(), E), nf4_expert_plan(r.experts, E)):
        assert torch.equal(got.cpu(), want) and torch.equal(plan, got)


def test_plan_where_one_expert_takes_all():
    """Runs of 8192 choices of one expert, several to a thread that adds them up."""
    e = torch.full((76800, 64), 63, dtype=torch.int32)
    e[40000:40003] = 62
    for got, want in zip(nf4_expert_plan(e.to(DEV), 64), sorted_plan(e, 64)):
        assert torch.equal(got.cpu(), want)


def test_route_of_no_tokens():
    r = nf4_route(torch.empty((0, 16), device=DEV), 4)
    assert r.weights.shape == (0, 4) and r.tokens.numel() == 0 and r.offsets.tolist() == [0] * 17
    assert nf4_expert_gather(torch.empty((0, 8), device=DEV), r).shape == (0, 8)
    assert nf4_expert_combine(torch.empty((0, 8), device=DEV), r).shape == (0, 8)


def routing(seed, T, E, k, empty=0):
    e = R.random_experts(seed, T, E, k, empty)
    w = torch.where(e >= 0, R.normal(seed + 1, T, k), torch.tensor(math.nan))      # the weight of nobody is not read
    host = NF4Routing(w, e, *R.plan(e, E))
    return host, NF4Routing(*(t.to(DEV) for t in (host.weights, host.experts, host.offsets, host.tokens, host.slots)))


ROWS = [(1, 1, 1, 1, 0), (3, 4, 2, 8, 1), (5, 8, 3, 7, 0), (33, 16, 8, 64, 3), (17, 64, 8, 2048, 0), (9, 8, 2, 2049, 2),
        (4, 64, 6, 5120, 1), (2, 4, 1, 20000, 0), (40, 5, 4, 12, 39), (6, 64, 64, 136, 0), (3, 3, 3, 16390, 1)]


@pytest.mark.parametrize("T,E,k,H,empty", ROWS)
@pytest.mark.parametrize("dtype", R.BOTH)
def test_gather(T, E, k, H, empty, dtype):
    host, r = routing(T + H, T, E, k, empty)
    x = R.normal(H, T, H).to(dtype)
    leaf = x.to(DEV).requires_grad_()
    rows = nf4_expert_gather(leaf, r)
    want = torch.zeros((T * k, H), dtype=dtype)
    n = int(host.offsets[-1])
    want[:n] = x[host.tokens[:n].long()]
    assert torch.equal(rows.detach().cpu(), want)
    g = R.normal(H + 1, T * k, H).to(dtype)
    g[n:] = math.nan                                            # rows of nobody are not read
    got, = torch.autograd.grad(rows, leaf, g.to(DEV))
    each = torch.where(host.slots[..., None] >= 0, g.double()[host.slots.clamp(min=0).long()], 0.0)
    s, size = each.sum(1), each.abs().sum(1)
    R.within(got, s, R.rounded(k * R.U32 * size, s, dtype))
    assert torch.equal(got, nf4_expert_gather_bwd(g.to(DEV), r))
    out = torch.full((T * k, H), 7.0, dtype=dtype, device=DEV)
    assert nf4_expert_gather(x.to(DEV), r, out=out) is out
    assert torch.equal(out[:n].cpu(), want[:n]) and bool((out[n:] == 7).all())


@pytest.mark.parametrize("T,E,k,H,empty", ROWS)
@pytest.mark.parametrize("dtype", R.BOTH)
def test_combine(T, E, k, H, empty, dtype):
    host, r = routing(T + H + 5, T, E, k, empty)
    n = int(host.offsets[-1])
    y = R.normal(H + 2, T * k, H).to(dtype)
    y[n:] = math.nan
    leaf, w = y.to(DEV).requires_grad_(), r.weights.clone().requires_grad_()
    out = nf4_expert_combine(leaf, NF4Routing(w, r.experts, r.offsets, r.tokens, r.slots))
    there = host.slots >= 0
    each = torch.where(there[..., None], y.double()[host.slots.clamp(min=0).long()], 0.0)
    weight = torch.where(there, host.weights.double(), 0.0)
    s, size = (each * weight[..., None]).sum(1), (each * weight[..., None]).abs().sum(1)
    R.within(out, s, R.rounded((k + 1) * R.U32 * size, s, dtype), "out")
    g = R.normal(H + 3, T, H).to(dtype)
    gy, gw = torch.autograd.grad(out, (leaf, w), g.to(DEV))
    dot, dots = (each * g.double()[:, None]).sum(-1), (each * g.double()[:, None]).abs().sum(-1)
    R.within(gw, dot, (H + 2) * R.U32 * dots + 1e-38, "grad_weights")
    want = torch.zeros((T * k, H), dtype=torch.float64)
    tok, j = there.nonzero(as_tuple=True)
    want[host.slots[tok, j].long()] = weight[tok, j][:, None] * g.double()[tok]
    R.within(gy, want, R.rounded(R.U32 * want.abs(), want, dtype), "grad_rows")
    assert bool((gy[n:] == 0).all())
    both = nf4_expert_combine_bwd(g.to(DEV), leaf.detach(), r)
    assert torch.equal(both[0], gy) and torch.equal(both[1], gw)
    into = torch.empty((T, H), dtype=dtype, device=DEV)
    assert nf4_expert_combine(leaf.detach(), r, out=into) is into and torch.equal(into, out.detach())


@pytest.mark.parametrize("which", [(True, False), (False, True)])
def test_combine_gradient_of_one_input(which):
    _, r = routing(3, 20, 8, 2, 2)
    y, g = R.normal(4, 40, 96).to(DEV), R.normal(5, 20, 96).to(DEV)
    both = nf4_expert_combine_bwd(g, y, r)
    leaf, w = y.clone().requires_grad_(which[0]), r.weights.clone().requires_grad_(which[1])
    nf4_expert_combine(leaf, NF4Routing(w, r.experts, r.offsets, r.tokens, r.slots)).backward(g)
    for have, got, want in zip(which, (leaf.grad, w.grad), both):
        assert (got is not None) == have and (not have or torch.equal(got, want))


def test_rows_of_other_types_strides_and_broadcast_gradients():
    host, r = routing(6, 21, 8, 2, 1)
    x = R.normal(7, 21, 200).to(DEV)
    for piece in (x[:, 8:136], x[:, 3:131], x.t().contiguous().t()[:, :128], x.half()[:, :128], x.double()[:, :128]):
        leaf = piece.detach().requires_grad_()
        rows = nf4_expert_gather(leaf, r)
        want = nf4_expert_gather(piece.float().contiguous(), r)
        assert rows.dtype == piece.dtype and torch.equal(rows.float(), want.to(piece.dtype).float())
        rows.sum().backward()                                   # its gradient is one number, broadcast
        count = (host.slots >= 0).sum(-1).to(DEV)
        assert leaf.grad.shape == leaf.shape and torch.equal(leaf.grad.float(), count[:, None].float().expand(21, 128))
        y = rows.detach().requires_grad_()
        nf4_expert_combine(y, r).sum().backward()
        assert y.grad.dtype == piece.dtype and y.grad.shape == y.shape
    big = torch.randn(21, 400, device=DEV)[:, :128]             # grad_out with strided rows
    assert torch.equal(nf4_expert_combine_bwd(big, want, r)[0], nf4_expert_combine_bwd(big.contiguous(), want, r)[0])
    odd = torch.empty(21 * 128 + 1, device=DEV)[1:].view(21, 128).copy_(x[:, :128])      # not 16-byte aligned
    assert torch.equal(nf4_expert_gather(odd, r), nf4_expert_gather(x[:, :128].contiguous(), r))


def test_malformed_slots_stay_in_range():
    """Slots outside the rows are choices without a row."""
    _, r = routing(8, 10, 4, 2)
    bad = r.slots.clone()
    bad[0, 0], bad[1, 1], bad[2, 0] = 20, 2 ** 31 - 1, -5
    x, y = R.normal(1, 10, 64).to(DEV), R.normal(2, 20, 64).to(DEV)
    s = NF4Routing(r.weights, r.experts, r.offsets, r.tokens, bad)
    none = NF4Routing(r.weights, r.experts, r.offsets, r.tokens, torch.where((bad < 0) | (bad >= 20), -1, bad))
    assert torch.equal(nf4_expert_combine(y, s), nf4_expert_combine(y, none))
    a, b = nf4_expert_gather(x, s, out=torch.zeros(20, 64, device=DEV)), nf4_expert_gather(x, none, out=torch.zeros(20, 64, device=DEV))
    assert torch.equal(a, b)
    assert torch.equal(nf4_expert_combine_bwd(x, y, s)[1], nf4_expert_combine_bwd(x, y, none)[1])


def test_results_repeat_bitwise():
    l = R.normal(1, 3000, 64).to(DEV)
    one, two = nf4_route(l, 8, bias=torch.zeros(64, device=DEV)), nf4_route(l, 8, bias=torch.zeros(64, device=DEV))
    for n in ("weights", "experts", "offsets", "tokens", "slots"):
        assert torch.equal(getattr(one, n), getattr(two, n))
    y = R.normal(2, 24000, 64).to(DEV)
    assert torch.equal(nf4_expert_combine_bwd(l, y, one)[1], nf4_expert_combine_bwd(l, y, two)[1])


def test_refusals_on_the_device():
    l = torch.zeros((4, 16), device=DEV)
    r = nf4_route(l, 2)
    leaf = torch.zeros(16, device=DEV, requires_grad=True)
    with pytest.raises(ValueError, match="bias requires a gradient"):
        nf4_route(l, 2, bias=leaf)
    for kw, what in ((dict(top_k=17), "top_k"), (dict(top_k=0), "top_k"), (dict(top_k=2, groups=3), "groups"),
                     (dict(top_k=2, groups=4, top_groups=5), "top_groups"), (dict(top_k=2, scale=0.0), "scale"),
                     (dict(top_k=2, scale=math.nan), "scale"), (dict(top_k=2, score="tanh"), "score"),
                     (dict(top_k=2, group_score="mean"), "group_score"), (dict(top_k=2, bias=torch.zeros(15, device=DEV)), "bias"),
                     (dict(top_k=2, bias=torch.zeros(16)), "bias"), (dict(top_k=2.5), "top_k")):
        with pytest.raises(ValueError, match=what):
            nf4_route(l, **kw)
    with pytest.raises(NF4Error):
        nf4_route(torch.zeros((2, 1025), device=DEV), 2)
    with pytest.raises(ValueError, match="floating"):
        nf4_route(l.int(), 2)
    x = torch.zeros((4, 8), device=DEV)
    with pytest.raises(ValueError, match="5 rows"):
        nf4_expert_gather(torch.zeros((5, 8), device=DEV), r)
    with pytest.raises(ValueError, match="rows must be"):
        nf4_expert_combine(x, r)
    with pytest.raises(ValueError, match="out"):
        nf4_expert_gather(x.requires_grad_(), r, out=torch.zeros((8, 8), device=DEV))
    with pytest.raises(ValueError, match="out must be"):
        nf4_expert_gather(x.detach(), r, out=torch.zeros((8, 8), device=DEV, dtype=torch.bfloat16))
    y = nf4_expert_gather(x, r)
    with pytest.raises(RuntimeError, match="not differentiable"):
        torch.autograd.grad(y.sum(), x, create_graph=True)
