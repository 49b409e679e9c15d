"""Ways of calling the expert and integer operators that their documentation allows:
without tokens or elements in training, under inference mode, from several
threads, with parts of a result kept alone, and each call in a graph of its own."""

import copy
import io
import threading

import pytest
import torch

import expert_ref as R
from nf4_bit_weight_amd import (NF4Int8, NF4Routing, nf4_expert_combine, nf4_expert_combine_bwd, nf4_expert_gather, nf4_expert_gather_bwd,
                                nf4_expert_plan, nf4_int8_grouped_matmul, nf4_int8_matmul, nf4_int8_quantize, nf4_route, nf4_route_bwd)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.mark.parametrize("T,H", [(0, 64), (0, 0), (5, 0)])
def test_empty_sizes_in_training(T, H):
    l, x = torch.zeros((T, 16), device=DEV, requires_grad=True), torch.zeros((T, H), device=DEV, requires_grad=True)
    r = nf4_route(l, 2, score="sigmoid")
    rows = nf4_expert_gather(x, r)
    y = nf4_expert_combine(rows, r)
    assert rows.shape == (2 * T, H) and y.shape == (T, H)
    gl, gx = torch.autograd.grad(y.sum() + r.weights.sum(), (l, x))
    assert gl.shape == l.shape and gx.shape == x.shape
    want = torch.sigmoid(torch.zeros(1)).item() ** 2
    assert torch.allclose(gl[:, :2], torch.full_like(gl[:, :2], want))       # of the weights' sum alone
    gr, gw = nf4_expert_combine_bwd(y.detach(), rows.detach(), r)
    assert gr.shape == rows.shape and gw.shape == (T, 2) and not gw.any()


def test_under_inference_mode():
    l, x = R.normal(1, 40, 64).to(DEV), R.normal(2, 40, 128).to(DEV)
    w = nf4_int8_quantize(R.normal(3, 64, 128).to(DEV))

    def run():
        r = nf4_route(l, 4)
        rows = nf4_expert_gather(x, r)
        return [r.weights, r.experts, r.offsets, r.tokens, r.slots, rows, nf4_expert_combine(rows, r), nf4_int8_matmul(x, w),
                *nf4_expert_plan(r.experts, 64)]
    want = run()
    with torch.inference_mode():
        got = run()
        assert all(t.is_inference() for t in got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_parts_of_a_routing_are_tensors_of_their_own():
    """Changed, copied or saved by itself, none of the four integer results touches another."""
    r = nf4_route(R.normal(1, 33, 16).to(DEV), 3)
    names = ("experts", "offsets", "tokens", "slots")
    want = {n: getattr(r, n).cpu() for n in names}
    for n in names:
        before = {m: getattr(r, m)._version for m in names}
        getattr(r, n).add_(1)
        assert {m for m in names if getattr(r, m)._version != before[m]} == {n}
        assert all(torch.equal(getattr(r, m).cpu(), want[m]) for m in names if m != n)
        getattr(r, n).sub_(1)
        assert getattr(r, n).is_contiguous() and torch.equal(copy.deepcopy(getattr(r, n)).cpu(), want[n])
        file = io.BytesIO()
        torch.save(getattr(r, n), file)
        file.seek(0)
        assert torch.equal(torch.load(file, weights_only=True).cpu(), want[n])


def test_threads_side_by_side():
    l, x = R.normal(1, 900, 64).to(DEV), R.normal(2, 900, 256).to(DEV)
    w = nf4_int8_quantize(R.normal(3, 64 * 96, 256).to(DEV)).per_expert(64)

    def run():
        leaf = l.clone().requires_grad_()
        r = nf4_route(leaf, 8, bias=torch.zeros(64, device=DEV))
        with torch.no_grad():
            y = nf4_int8_grouped_matmul(x, r.offsets, w, 64, tokens=r.tokens)
        out = nf4_expert_combine(y, r)
        return [r.slots, y, out.detach(), *torch.autograd.grad(out.sum(), leaf)]
    want = run()
    torch.cuda.synchronize()
    got, failed = [], []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    got.append(run())
            s.synchronize()
        except Exception as e:                                  # seen below, in the test's own thread
            failed.append(e)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and len(got) == 20
    assert all(torch.equal(a, b) for outs in got for a, b in zip(outs, want))


def cases():
    host = R.random_experts(5, 300, 16, 4, 9)
    e = host.to(DEV)
    off, tok, slot = (t.to(DEV) for t in R.plan(host, 16))
    r = NF4Routing(torch.rand(300, 4, device=DEV), e, off, tok, slot)
    x, y, l = torch.empty(300, 130, device=DEV), torch.empty(1200, 130, device=DEV), torch.empty(300, 16, device=DEV)
    g = torch.empty(300, 4, device=DEV)
    w = nf4_int8_quantize(R.normal(6, 16 * 48, 130).to(DEV))
    plain = NF4Int8(w.q, w.scale, w.N, w.K)
    return [x, y, l, g], {
        "plan": lambda: nf4_expert_plan(e, 16),
        "gather": lambda: [nf4_expert_gather(x, r)],
        "gather_bwd": lambda: [nf4_expert_gather_bwd(y, r)],
        "combine": lambda: [nf4_expert_combine(y, r)],
        "combine_bwd": lambda: nf4_expert_combine_bwd(x, y, r),
        "route": lambda: vars(nf4_route(l, 4, groups=4, top_groups=2, group_score="top2")).values(),
        "route_bwd": lambda: [nf4_route_bwd(g, l, r)],
        "quantize": lambda: [nf4_int8_quantize(x).q, nf4_int8_quantize(x).scale],
        "matmul": lambda: [nf4_int8_matmul(x, plain), nf4_int8_matmul(x[:2], plain), nf4_int8_matmul(nf4_int8_quantize(x), plain)],
        "grouped": lambda: [nf4_int8_grouped_matmul(x, off, w.per_expert(16), 16, tokens=tok), nf4_int8_grouped_matmul(y, off, w.per_expert(16), 16)],
    }


@pytest.mark.parametrize("name", ["plan", "gather", "gather_bwd", "combine", "combine_bwd", "route", "route_bwd", "quantize", "matmul", "grouped"])
def test_each_call_replays_from_a_graph(name):
    inputs, calls = cases()
    f = calls[name]

    def fresh(seed):
        for i, t in enumerate(inputs):
            t.copy_(R.normal(10 * seed + i, *t.shape))
    fresh(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = list(f())
    for i in range(1, 4):
        fresh(i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = list(f())
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {i}"
