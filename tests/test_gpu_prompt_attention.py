"""Causal attention over packed prompts on the GPU, forward and backward."""

import numpy as np
import pytest
import torch

import attn_ref as R
from nf4_bit_weight_amd import (api, nf4_prompt_attention, nf4_prompt_attention_bwd, nf4_prompt_attention_fwd)

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
LENS = [[1], [2, 0, 63], [64, 65], [127, 1, 128], [129, 300], [31, 33, 0, 0, 5, 200]]


def inputs(lens, Hq, Hkv, D, seed=0, extra=0):
    T = sum(lens) + extra
    joint = R.normal(seed, T, Hq + 2 * Hkv, D)
    return joint, joint[:, :Hq], joint[:, Hq:Hq + Hkv], joint[:, Hq + Hkv:]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", LENS)
def test_forward(lens, D):
    Hq, Hkv = 6, 2
    joint, q, k, v = inputs(lens, Hq, Hkv, D, seed=sum(lens))
    jd = joint.to(DEV)                                          # rows of a joint projection, taken as they are
    off = R.offsets_of(lens).to(DEV)
    out, _, lse = nf4_prompt_attention_fwd(jd[:, :Hq], jd[:, Hq:Hq + Hkv], jd[:, Hq + Hkv:], off, for_backward=True)
    sc = float(np.float32(D ** -0.5))
    want, bound = R.prompt(q, k, v, lens, sc)["out"]
    R.within(out, want, bound, f"{lens}")
    at = 0
    for n in lens:
        if n:
            qs, ks = q[at:at + n].double(), k[at:at + n].double().repeat_interleave(3, 1)
            s = torch.einsum("thd,shd->hts", qs, ks) * sc
            s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -np.inf)
            w = torch.logsumexp(s, -1)
            # the sum's n terms and the score's D products in fp32, logarithm and sum within 2^-20 of their size
            assert ((lse[:, at:at + n].cpu().double() - w).abs() <= 2.0 ** -20 * (w.abs() + 8) + (n + 40 * D) * R.F).all()
        at += n


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (5, 1), (16, 2)])
def test_forward_heads(Hq, Hkv):
    lens = [70, 9]
    _, q, k, v = inputs(lens, Hq, Hkv, 64, seed=Hq)
    out = nf4_prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), R.offsets_of(lens).to(DEV))
    R.within(out, *R.prompt(q, k, v, lens, 0.125)["out"], f"{Hq}/{Hkv}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", LENS)
def test_backward(lens, D):
    Hq, Hkv = 4, 2
    _, q, k, v = inputs(lens, Hq, Hkv, D, seed=7 + sum(lens))
    gy = R.normal(99, sum(lens), Hq, D)
    leaves = [x.to(DEV).contiguous().requires_grad_() for x in (q, k, v)]
    out = nf4_prompt_attention(*leaves, R.offsets_of(lens).to(DEV))
    grads = torch.autograd.grad(out, leaves, gy.to(DEV))
    want = R.prompt(q, k, v, lens, float(np.float32(D ** -0.5)), gy)
    R.within(out, *want["out"], f"{lens} out")
    for name, g in zip(("grad_q", "grad_k", "grad_v"), grads):
        R.within(g, *want[name], f"{lens} {name}")


@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (7, 1), (16, 2)])
def test_backward_heads(Hq, Hkv):
    lens = [70, 9]
    _, q, k, v = inputs(lens, Hq, Hkv, 128, seed=Hq)
    gy = R.normal(98, sum(lens), Hq, 128)
    leaves = [x.to(DEV).contiguous().requires_grad_() for x in (q, k, v)]
    grads = torch.autograd.grad(nf4_prompt_attention(*leaves, R.offsets_of(lens).to(DEV), 0.2), leaves, gy.to(DEV))
    want = R.prompt(q, k, v, lens, float(np.float32(0.2)), gy)
    for name, g in zip(("grad_q", "grad_k", "grad_v"), grads):
        R.within(g, *want[name], f"{Hq}/{Hkv} {name}")


def test_backward_against_differences():
    """The kernel's gradients along random directions against central
    differences of the 64-bit forward."""
    lens, Hq, Hkv, D = [20, 37], 4, 2, 64
    _, q, k, v = inputs(lens, Hq, Hkv, D, seed=4)
    gy = R.normal(97, sum(lens), Hq, D)
    leaves = [x.to(DEV).contiguous().requires_grad_() for x in (q, k, v)]
    grads = torch.autograd.grad(nf4_prompt_attention(*leaves, R.offsets_of(lens).to(DEV)), leaves, gy.to(DEV))
    bounds = R.prompt(q, k, v, lens, 0.125, gy)
    base = [x.double() for x in (q, k, v)]
    eps = 1e-4
    for i, name in enumerate(("grad_q", "grad_k", "grad_v")):
        d = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)

        def f(x):
            args = list(base)
            args[i] = base[i] + x * d
            return float((R.prompt(*args, lens, 0.125)["out"][0] * gy.double()).sum())

        diff = (f(eps) - f(-eps)) / (2 * eps)
        got = float((grads[i].cpu().double() * d).sum())
        # the bound of every element along the direction; the difference's own error is of order eps^2
        room = float((bounds[name][1] * d.abs()).sum()) + 1e-4 * (abs(diff) + 1)
        assert abs(got - diff) <= room, (name, got, diff, room)


def test_long_row_of_keys():
    """Many tiles, more sequences than a wave has lanes."""
    lens = [3] * 70 + [1500] + [0] * 5 + [40]
    Hq, Hkv, D = 2, 1, 128
    _, q, k, v = inputs(lens, Hq, Hkv, D, seed=12)
    gy = R.normal(96, sum(lens), Hq, D)
    leaves = [x.to(DEV).contiguous().requires_grad_() for x in (q, k, v)]
    out = nf4_prompt_attention(*leaves, R.offsets_of(lens).to(DEV))
    grads = torch.autograd.grad(out, leaves, gy.to(DEV))
    want = R.prompt(q, k, v, lens, float(np.float32(D ** -0.5)), gy)
    R.within(out, *want["out"], "out")
    for name, g in zip(("grad_q", "grad_k", "grad_v"), grads):
        R.within(g, *want[name], name)


def test_large_scores():
    """Scores of hundreds: the running maximum carries the softmax."""
    lens = [150]
    _, q, k, v = inputs(lens, 2, 2, 64, seed=5)
    q = (q.float() * 30).to(torch.bfloat16)
    out = nf4_prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), R.offsets_of(lens).to(DEV))
    R.within(out, *R.prompt(q, k, v, lens, 0.125)["out"], "large scores")


@pytest.mark.parametrize("at", [0, 40, 63, 64, 100, 199])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_odd_values_reach_only_their_readers(at, value):
    """A key or value that is no number leaves the rows before its token alone."""
    lens, D = [200], 128
    _, q, k, v = inputs(lens, 2, 1, D, seed=6)
    want, bound = R.prompt(q, k, v, lens, float(np.float32(D ** -0.5)))["out"]
    off = R.offsets_of(lens).to(DEV)
    v2 = v.clone()
    v2[at, 0, 5] = value
    out = nf4_prompt_attention(q.to(DEV), k.to(DEV), v2.to(DEV), off)
    R.within(out[:at], want[:at], bound[:at], "rows before")
    assert not torch.isfinite(out[at:, :, 5]).any()
    other = torch.arange(D) != 5
    R.within(out[:, :, other.to(DEV)], want[:, :, other], bound[:, :, other], "other elements")
    if value > 0:
        assert (out[at:, :, 5] == value).all()
    k2 = k.clone()
    k2[at, 0, 7] = float("nan")
    out = nf4_prompt_attention(q.to(DEV), k2.to(DEV), v.to(DEV), off)
    R.within(out[:at], want[:at], bound[:at], "rows before")
    assert torch.isnan(out[at:]).all()


def test_rows_outside_sequences():
    """Padding that holds NaN reaches nothing; its results are zeros in fresh
    tensors, and as they were in one passed in."""
    lens, Hq, Hkv, D, pad = [30, 100], 2, 1, 64, 90
    _, q, k, v = inputs(lens, Hq, Hkv, D, extra=pad)
    T = sum(lens)
    for x in (q, k, v):
        x[T:] = float("nan")
    gy = R.normal(95, T + pad, Hq, D)
    gy[T:] = float("inf")
    off = R.offsets_of(lens).to(DEV)
    leaves = [x.to(DEV).contiguous().requires_grad_() for x in (q, k, v)]
    out = nf4_prompt_attention(*leaves, off)
    grads = torch.autograd.grad(out, leaves, gy.to(DEV))
    want = R.prompt(q[:T], k[:T], v[:T], lens, 0.125, gy[:T])
    R.within(out[:T], *want["out"], "out")
    for name, g in zip(("grad_q", "grad_k", "grad_v"), grads):
        R.within(g[:T], *want[name], name)
        assert not g[T:].any()
    assert not out[T:].any()
    mark = torch.full_like(out, 3.0).detach()
    o2 = nf4_prompt_attention_fwd(*(x.detach() for x in leaves), off, out=mark)
    assert torch.equal(o2[:T], out[:T]) and (o2[T:] == 3.0).all()


def test_no_sequences():
    q = R.normal(1, 5, 2, 64).to(DEV)
    out = nf4_prompt_attention(q, q, q, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert not out.any()
    none = q[:0]
    leaves = [none.clone().requires_grad_() for _ in range(3)]
    out = nf4_prompt_attention(*leaves, torch.zeros(3, dtype=torch.int32, device=DEV))
    out.sum().backward()
    assert out.shape == (0, 2, 64) and leaves[0].grad.shape == (0, 2, 64)


def test_other_dtypes_and_grad_layouts():
    """fp32 and fp16 callers get their own type back; an expanded or transposed
    output gradient is taken; only the wanted gradients are returned."""
    lens, H, D = [40, 25], 2, 64
    _, q, k, v = inputs(lens, H, H, D, seed=3)
    off = R.offsets_of(lens).to(DEV)
    ref = [x.to(DEV).contiguous().requires_grad_() for x in (q, k, v)]
    out = nf4_prompt_attention(*ref, off)
    gy = R.normal(94, sum(lens), H, D).to(DEV)
    base = torch.autograd.grad(out, ref, gy, retain_graph=True)
    for dt in (torch.float32, torch.float16):
        xs = [x.detach().to(dt).requires_grad_() for x in ref]
        o = nf4_prompt_attention(*xs, off)
        gs = torch.autograd.grad(o, xs, gy.to(dt))
        assert o.dtype == dt and all(g.dtype == dt for g in gs)
        if dt is torch.float32:                                  # bf16 values pass through fp32 unchanged
            assert torch.equal(o, out.to(dt)) and all(torch.equal(a, b.to(dt)) for a, b in zip(gs, base))
    strange = gy.transpose(0, 1).contiguous().transpose(0, 1)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(out, ref, strange, retain_graph=True), base))
    ones = torch.autograd.grad(out.sum(), ref, retain_graph=True)
    want = torch.autograd.grad(out, ref, torch.ones_like(out))
    assert all(torch.equal(a, b) for a, b in zip(ones, want))
    frozen = [ref[0].detach(), ref[1].detach(), ref[2].detach().requires_grad_()]
    nf4_prompt_attention(*frozen, off).backward(gy)
    assert frozen[0].grad is None and torch.equal(frozen[2].grad, base[2])


def test_shared_leaf_and_checkpoint():
    """One tensor as q, k and v adds its three gradients; recomputation under
    activation checkpointing gives the same bits."""
    from torch.utils.checkpoint import checkpoint

    lens = [33, 70]
    off = R.offsets_of(lens).to(DEV)
    x = R.normal(8, sum(lens), 2, 64).to(DEV).requires_grad_()
    gy = R.normal(93, sum(lens), 2, 64).to(DEV)
    three = [x.detach().clone().requires_grad_() for _ in range(3)]
    g3 = torch.autograd.grad(nf4_prompt_attention(*three, off), three, gy)
    (g,) = torch.autograd.grad(nf4_prompt_attention(x, x, x, off), x, gy)
    # bf16 sums of three terms: at most two roundings of the running sum
    want = sum(t.double() for t in g3)
    room = 2 * R.U * sum(t.double().abs() for t in g3)
    assert ((g.double() - want).abs() <= room).all()
    y = checkpoint(lambda a: nf4_prompt_attention(a, a, a, off), x, use_reentrant=False)
    (gc,) = torch.autograd.grad(y, x, gy)
    assert torch.equal(gc, g)


def test_saved_tensors_and_second_order():
    """What the node saves goes through the saved-tensor hooks, an operand
    changed in place is noticed, and a second derivative is refused."""
    lens = [20]
    off = R.offsets_of(lens).to(DEV)
    xs = [R.normal(i, 20, 2, 64).to(DEV).requires_grad_() for i in range(3)]
    seen = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (seen.append(t.shape), t.clone())[1], lambda t: t):
        out = nf4_prompt_attention(*xs, off)
    assert len(seen) == 7
    ref = torch.autograd.grad(nf4_prompt_attention(*xs, off), xs, torch.ones_like(out))
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(out, xs, torch.ones_like(out)), ref))
    out = nf4_prompt_attention(*xs, off)
    with pytest.raises(RuntimeError, match="not differentiable"):
        torch.autograd.grad(out, xs, torch.ones_like(out), create_graph=True)
    out = nf4_prompt_attention(*xs, off)
    with torch.no_grad():
        xs[1].add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_repeatable_and_streams():
    lens = [300, 1, 500]
    _, q, k, v = inputs(lens, 8, 2, 128, seed=2)
    off = R.offsets_of(lens).to(DEV)
    xs = [x.to(DEV).contiguous() for x in (q, k, v)]
    gy = R.normal(92, sum(lens), 8, 128).to(DEV)
    out, rest, lse = nf4_prompt_attention_fwd(*xs, off, for_backward=True)
    ref = nf4_prompt_attention_bwd(gy, *xs, out, rest, lse, off)
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            o, r, l = nf4_prompt_attention_fwd(*xs, off, for_backward=True)
            g = nf4_prompt_attention_bwd(gy, *xs, o, r, l, off)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse) and all(torch.equal(a, b) for a, b in zip(g, ref))


def test_graph_follows_the_offsets():
    """A captured forward and backward replayed with other lengths."""
    T, Hq, Hkv, D = 160, 4, 2, 64
    _, q, k, v = inputs([T], Hq, Hkv, D, seed=1)
    xs = [x.to(DEV).contiguous() for x in (q, k, v)]
    gy = R.normal(91, T, Hq, D).to(DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)

    def step():
        o, r, l = nf4_prompt_attention_fwd(*xs, off, for_backward=True)
        return (o, *nf4_prompt_attention_bwd(gy, *xs, o, r, l, off))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for lens in ([160, 0, 0], [40, 50, 70], [0, 1, 100], [1, 129, 30]):
        off.copy_(R.offsets_of(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step())), lens


def test_path_counts_and_refusals():
    x = R.normal(1, 6, 2, 64).to(DEV)
    off = torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    api.nf4_reset_path_counts()
    out, rest, lse = nf4_prompt_attention_fwd(x, x, x, off, for_backward=True)
    nf4_prompt_attention_bwd(x, x, x, x, out, rest, lse, off)
    c = api.nf4_path_counts()
    assert (c["prompt_fwd"], c["prompt_bwd"]) == (1, 1)

    def bad(*a, **kw):
        with pytest.raises(ValueError):
            nf4_prompt_attention_fwd(*a, **kw)

    bad(x, x, x, off.long())
    bad(x, x, x, off.cpu())
    bad(x, x, x, off[:0])
    bad(x.float(), x, x, off)
    bad(x, x[:5], x, off)
    bad(x[:, :1], x, x, off)
    bad(x, x[:, :1], x, off)
    bad(x[..., :32], x[..., :32], x[..., :32], off)
    bad(x, x, x, off, scale=-1.0)
    bad(x, x, x, off, out=x.float())
    with pytest.raises(ValueError):
        nf4_prompt_attention_bwd(x, x, x, x, out, rest, lse[:1], off)
    with pytest.raises(RuntimeError):
        nf4_prompt_attention_bwd(x, x, x, x, out, rest, lse, off, ws=torch.empty(16, dtype=torch.uint8, device=DEV))


def leaves():
    _, q, k, v = inputs([100], 4, 2, 64, seed=5)
    return [x.to(DEV).contiguous().requires_grad_() for x in (q, k, v)]


def test_captured_step_of_leaves():
    """Forward and backward through autograd, captured and replayed on changed
    inputs."""
    xs, off = leaves(), torch.tensor([0, 37, 100], dtype=torch.int32, device=DEV)
    gy = R.normal(93, 100, 4, 64).to(DEV)

    def step(xs):
        y = nf4_prompt_attention(*xs, off)
        return (y.detach(), *torch.autograd.grad(y, xs, gy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(xs)
    for seed in range(3):
        with torch.no_grad():
            for i, x in enumerate(xs):
                x.copy_(R.normal(200 + 3 * seed + i, *x.shape))
        graph.replay()
        torch.cuda.synchronize()
        want = step([x.detach().requires_grad_() for x in xs])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_capture_refuses_leaves_of_a_living_eager_graph():
    xs, off = leaves(), torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    alive = nf4_prompt_attention(*xs, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="eager graph"):
            nf4_prompt_attention(*xs, off)
        with torch.no_grad():
            out = nf4_prompt_attention(*xs, off)               # no backward pass, no accumulators
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, alive.detach())
    grads = torch.autograd.grad(alive, xs, torch.ones_like(alive))
    assert all(g.isfinite().all() for g in grads)


@pytest.mark.parametrize("lens", [[1], [1] * 8, [1, 40, 1, 129]])
@pytest.mark.parametrize("Hq,Hkv,D", [(12, 4, 64), (4, 4, 128)])
def test_a_single_key_has_no_score_gradient(lens, Hq, Hkv, D):
    """A row that sees one key weighs it with 1: exactly no gradient reaches its
    query, and its key gets none from it."""
    _, q, k, v = inputs(lens, Hq, Hkv, D, seed=11)
    off = R.offsets_of(lens).to(DEV)
    xs = [x.to(DEV).contiguous().requires_grad_() for x in (q, k, v)]
    gy = R.normal(95, sum(lens), Hq, D).to(DEV)
    gq, gk, gv = torch.autograd.grad(nf4_prompt_attention(*xs, off), xs, gy)
    first = off[:-1].long()
    assert not gq[first].any()
    alone = first[torch.tensor([n == 1 for n in lens], device=DEV)]
    assert not gk[alone].any()
    # grad_v there is the sum of the group's output gradients, rounded once
    want = gy[alone].double().unflatten(1, (Hkv, Hq // Hkv))
    room = (R.U + 2.0 ** -20) * want.abs().sum(2)
    assert ((gv[alone].double() - want.sum(2)).abs() <= room).all()


def test_a_nan_score_of_a_single_key_is_not_hidden():
    _, q, k, v = inputs([1, 5], 2, 2, 64, seed=12)
    q[0, 0, 3] = float("nan")
    xs = [x.to(DEV).contiguous().requires_grad_() for x in (q, k, v)]
    off = R.offsets_of([1, 5]).to(DEV)
    out = nf4_prompt_attention(*xs, off)
    gq, _, _ = torch.autograd.grad(out, xs, torch.ones_like(out))
    assert out[0, 0].isnan().all() and gq[0, 0].isnan().all()
    assert out[1:].isfinite().all() and gq[1:].isfinite().all()
