"""The expert operators with the grouped projections between them, as a model
runs them: an expert layer forward and back through the quantised experts, the
same layer served in 8-bit integers, and both captured into graphs."""

import pytest
import torch
from torch.utils.checkpoint import checkpoint

import expert_ref as R
import workloads as WL
from nf4_bit_weight_amd import (NF4Routing, nf4_expert_combine, nf4_expert_combine_bwd, nf4_expert_gather, nf4_expert_gather_bwd,
                                nf4_grouped_linear, nf4_grouped_matmul_bwd_input, nf4_grouped_matmul_fwd, nf4_int8_grouped_matmul,
                                nf4_int8_matmul, nf4_int8_quantize, nf4_quantize, nf4_route, nf4_route_bwd)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
T, E, K, HID, MID = 50, 8, 2, 256, 128
HOW = dict(score="sigmoid", renormalize=True, scale=1.5)


def stacks():
    code = torch.from_numpy(WL.nf4_code_np()).to(DEV)
    w = [WL.gpu_weight_f32(E * n, k, seed=500 + i, device=DEV, std=0.08) for i, (n, k) in enumerate(((MID, HID), (MID, HID), (HID, MID)))]
    return w, [nf4_quantize(x, code).per_expert(E) for x in w]


def router():
    return (0.2 * R.normal(9, E, HID)).to(DEV), (0.05 * R.normal(10, E)).to(DEV)


def layer(x, wr, bias, w):
    r = nf4_route(x.float() @ wr.t(), K, bias=bias, **HOW)
    rows = nf4_expert_gather(x, r)
    h = torch.nn.functional.silu(nf4_grouped_linear(rows, r.offsets, w[0], E)) * nf4_grouped_linear(rows, r.offsets, w[1], E)
    return nf4_expert_combine(nf4_grouped_linear(h, r.offsets, w[2], E), r), r


def inputs(seed=1):
    return R.normal(seed, T, HID).to(torch.bfloat16).to(DEV), R.normal(seed + 1, T, HID).to(torch.bfloat16).to(DEV)


def test_layer_forward_and_back_are_its_calls():
    """The gradients are the calls' own, one behind the other."""
    _, w = stacks()
    wr, bias = router()
    x, gy = inputs()
    leaf, wrl = x.clone().requires_grad_(), wr.clone().requires_grad_()
    y, r = layer(leaf, wrl, bias, w)
    y.backward(gy)

    logits = x.float() @ wr.t()
    s = nf4_route(logits, K, bias=bias, **HOW)
    assert torch.equal(s.weights, r.weights.detach()) and torch.equal(s.slots, r.slots)
    rows = nf4_expert_gather(x, s)
    g, u = (nf4_grouped_matmul_fwd(rows, s.offsets, w[i], E) for i in (0, 1))
    gl, ul = g.clone().requires_grad_(), u.clone().requires_grad_()
    h = torch.nn.functional.silu(gl) * ul
    d = nf4_grouped_matmul_fwd(h.detach(), s.offsets, w[2], E)
    assert torch.equal(nf4_expert_combine(d, s), y.detach())
    gd, gw = nf4_expert_combine_bwd(gy, d, s)
    h.backward(nf4_grouped_matmul_bwd_input(gd, s.offsets, w[2], E))
    grows = [nf4_grouped_matmul_bwd_input(t.grad, s.offsets, w[i], E) for i, t in enumerate((gl, ul))]
    glog = nf4_route_bwd(gw, logits, s, **HOW)
    direct = nf4_expert_gather_bwd(grows[0] + grows[1], s)
    # the two ways to x come together in bf16
    parts = [direct.double(), (glog @ wr).double()]
    assert ((leaf.grad.double() - sum(parts)).abs() <= 2 * R.U[torch.bfloat16] * sum(p.abs() for p in parts) + 1e-30).all()
    # a product of fp32 matrices over T rows, taken twice by the same library
    assert ((wrl.grad - glog.t() @ x.float()).abs() <= 2 * T * R.U32 * (glog.abs().t() @ x.float().abs()) + 1e-30).all()


def test_layer_under_checkpointing():
    _, w = stacks()
    wr, bias = router()
    x, gy = inputs(3)
    grads = []
    for wrapped in (False, True):
        leaf = x.clone().requires_grad_()
        f = lambda t: layer(t, wr, bias, w)[0]
        y = checkpoint(f, leaf, use_reentrant=False) if wrapped else f(leaf)
        y.backward(gy)
        grads.append((y.detach(), leaf.grad))
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])


def test_padding_tokens_pass_through_the_layer():
    """Tokens without experts come out as zeros, and no other token sees them."""
    _, w = stacks()
    wr, _ = router()
    x, gy = inputs(5)
    x[T - 7:] = float("nan")
    logits = (x.float() @ wr.t())
    logits[T - 7:] = -float("inf")

    def run(x, logits):
        leaf = x.clone().requires_grad_()
        r = nf4_route(logits, K)
        rows = nf4_expert_gather(leaf, r)
        y = nf4_expert_combine(nf4_grouped_linear(rows, r.offsets, w[0], E), r)
        y.backward(gy[: x.shape[0], :MID].contiguous())
        return y.detach(), leaf.grad
    y, g = run(x, logits)
    some, gs = run(x[: T - 7].contiguous(), logits[: T - 7].contiguous())
    assert torch.equal(y[: T - 7], some) and torch.equal(g[: T - 7], gs)
    assert bool((y[T - 7:] == 0).all()) and bool((g[T - 7:] == 0).all())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens,some", [(6, 3), (50, 43), (700, 300)])
def test_grouped_calls_leave_the_rows_of_nobody(bits, tokens, some):
    code = torch.from_numpy(WL.nf4_code_np() if bits == 4 else WL.int8_code_np()).to(DEV)
    w = nf4_quantize(WL.gpu_weight_f32(E * MID, HID, seed=510, device=DEV, std=0.08), code, bits=bits).per_expert(E)
    logits = R.normal(11, tokens, E).to(DEV)
    logits[some:] = -float("inf")
    r = nf4_route(logits, K)
    for f, n, m in ((nf4_grouped_matmul_fwd, HID, MID), (nf4_grouped_matmul_bwd_input, MID, HID)):
        rows = R.normal(12, tokens * K, n).to(torch.bfloat16).to(DEV)
        out = torch.full((tokens * K, m), 7.0, dtype=torch.bfloat16, device=DEV)
        f(rows, r.offsets, w, E, out)
        assert bool((out[some * K:] == 7).all()) and bool((out[: some * K] != 7).any(1).all())


def served(x, logits, w8):
    r = nf4_route(logits, K, **HOW)
    xq = nf4_int8_quantize(x)                                    # once for both projections
    g, u = (nf4_int8_grouped_matmul(xq, r.offsets, w8[i], E, tokens=r.tokens) for i in (0, 1))
    h = torch.nn.functional.silu(g) * u
    return nf4_expert_combine(nf4_int8_grouped_matmul(h, r.offsets, w8[2], E), r)


def test_layer_served_in_integers():
    """Each call of the layer against exact sums over what the call before it gave."""
    w, _ = stacks()
    w8 = [nf4_int8_quantize(x).per_expert(E) for x in w]
    wr, _ = router()
    x, _ = inputs(7)
    logits = x.float() @ wr.t()
    r = nf4_route(logits, K, **HOW)
    weights, experts = R.route(logits.cpu(), K, **HOW)
    assert torch.equal(r.experts.cpu(), experts)
    off, tok, slot = R.plan(experts, E)

    def check(y, rows, i):
        n = (MID, MID, HID)[i]
        q, s = R.quantize(rows)
        qw, sw = R.quantize(w[i].cpu())
        for e in range(E):
            a, b = int(off[e]), int(off[e + 1])
            want, bound = R.product(q[a:b], s[a:b], qw[e * n:(e + 1) * n], sw[e * n:(e + 1) * n])
            R.within(y[a:b], want, R.rounded(bound, want, torch.bfloat16), f"projection {i} expert {e}")
    xq = nf4_int8_quantize(x)
    g, u = (nf4_int8_grouped_matmul(xq, r.offsets, w8[i], E, tokens=r.tokens) for i in (0, 1))
    check(g, x.cpu()[tok.long()], 0)
    check(u, x.cpu()[tok.long()], 1)
    h = torch.nn.functional.silu(g) * u
    d = nf4_int8_grouped_matmul(h, r.offsets, w8[2], E)
    check(d, h.cpu(), 2)
    y = nf4_expert_combine(d, r)
    each = d.cpu().double()[slot.long()] * r.weights.cpu().double()[..., None]
    want, size = each.sum(1), each.abs().sum(1)
    R.within(y, want, R.rounded((K + 1) * R.U32 * size, want, torch.bfloat16), "combined")
    assert torch.equal(served(x, logits, w8), y)


def replay_check(capture, eager, fresh, rounds=3):
    """Replays on new inputs, with eager work between them, give the eager results."""
    for i in range(rounds):
        fresh(i)
        capture.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in eager.outputs]
        want = eager()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w), f"replay {i}"


class Eager:
    def __init__(self, f):
        self.f, self.outputs = f, None

    def __call__(self):
        return self.f()


@pytest.mark.parametrize("tokens", [1, T, 700])
def test_serving_calls_replay_from_a_graph(tokens):
    w, _ = stacks()
    w8 = [nf4_int8_quantize(x).per_expert(E) for x in w]
    wr, bias = router()
    dense = nf4_int8_quantize(R.normal(20, 300, HID).to(DEV))
    x = torch.zeros((tokens, HID), dtype=torch.bfloat16, device=DEV)
    logits = torch.zeros((tokens, E), device=DEV)

    def run():
        r = nf4_route(logits, K, bias=bias, **HOW)
        return [r.weights, r.experts, r.offsets, r.tokens, r.slots, nf4_expert_gather(x, r), served(x, logits, w8), nf4_int8_matmul(x, dense)]

    def fresh(i):
        x.copy_(R.normal(30 + i, tokens, HID))
        logits.copy_(R.normal(40 + i, tokens, E))
        if i == 1:
            logits[tokens // 2:] = -float("inf")                 # the rows behind the last expert's change from replay to replay
    fresh(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    e = Eager(run)
    with torch.cuda.graph(g):
        e.outputs = run()
    replay_check(g, e, fresh)


def test_training_step_replays_from_a_graph():
    _, w = stacks()
    wr, bias = router()
    x, gy = inputs(11)
    leaf = x.clone().requires_grad_()

    def run():
        r = nf4_route(leaf.float() @ wr.t(), K, bias=bias, **HOW)
        rows = nf4_expert_gather(leaf, r)
        y = nf4_expert_combine(nf4_grouped_linear(rows, r.offsets, w[0], E), r)
        return [y.detach(), *torch.autograd.grad(y, leaf, gy[:, :MID].contiguous())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    e = Eager(run)
    with torch.cuda.graph(g):
        e.outputs = run()

    def fresh(i):
        with torch.no_grad():
            leaf.copy_(R.normal(60 + i, T, HID))
    replay_check(g, e, fresh)


@pytest.mark.parametrize("call", ["route", "gather", "combine rows", "combine weights"])
def test_a_captured_call_refuses_a_leaf_whose_eager_graph_lives(call):
    r = nf4_route(R.normal(1, 12, E).to(DEV), K)
    rows = nf4_expert_gather(R.normal(2, 12, 64).to(DEV), r)
    leaf = {"route": R.normal(3, 12, E).to(DEV), "gather": R.normal(4, 12, 64).to(DEV), "combine rows": rows.clone(),
            "combine weights": r.weights.clone()}[call].requires_grad_()

    def run():
        if call == "route":
            return nf4_route(leaf, K).weights
        if call == "gather":
            return nf4_expert_gather(leaf, r)
        if call == "combine rows":
            return nf4_expert_combine(leaf, r)
        return nf4_expert_combine(rows, NF4Routing(leaf, r.experts, r.offsets, r.tokens, r.slots))
    alive = run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    refused = None
    with torch.cuda.graph(g):
        try:
            run()
        except ValueError as e:
            refused = str(e)
        torch.zeros(1, device=DEV)
    assert refused and "eager graph" in refused
    del alive


def test_calls_on_another_stream_and_two_at_once():
    """Work goes to the tensors' device's current stream; calls side by side do not meet."""
    logits, x = R.normal(1, 600, 64).to(DEV), R.normal(2, 600, 512).to(DEV)
    w8 = nf4_int8_quantize(R.normal(3, 700, 512).to(DEV))

    def run():
        r = nf4_route(logits, 8)
        rows = nf4_expert_gather(x, r)
        return [r.weights, r.tokens, r.slots, rows, nf4_expert_combine(rows, r), nf4_int8_matmul(x, w8), nf4_int8_matmul(x[:1], w8)]
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_forward_mode_tangents_are_refused():
    import torch.autograd.forward_ad as fwAD
    l, x = R.normal(1, 6, 8).to(DEV), R.normal(2, 6, 64).to(DEV)
    r = nf4_route(l, 2)
    w8 = nf4_int8_quantize(R.normal(3, 32, 64).to(DEV))
    with fwAD.dual_level():
        for f, t in ((lambda d: nf4_route(d, 2), l), (lambda d: nf4_expert_gather(d, r), x),
                     (lambda d: nf4_expert_combine(d, r), torch.cat((x, x))), (lambda d: nf4_int8_matmul(d, w8), x)):
            with pytest.raises(ValueError, match="tangent"):
                f(fwAD.make_dual(t, torch.ones_like(t)))
