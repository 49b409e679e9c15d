"""Host-side checks of the expert calls and of the products in 8-bit integers
(nf4_experts.h, nf4_int8.h): exports, what each call refuses, and the plain
forms that the GPU tests compare with.  No device work is issued: every call
here fails its checks or is empty."""

import ctypes
import math
import os
import re

import pytest
import torch

import expert_ref as R
from nf4_bit_weight_amd import (NF4Int8, NF4Routing, nf4_expert_combine, nf4_expert_gather, nf4_expert_plan, nf4_int8_matmul,
                                nf4_int8_quantize, nf4_route)
from nf4_bit_weight_amd import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, BAD = 0x10000, 0x10008          # aligned and not; never dereferenced
BIG = ctypes.c_size_t(-1).value
OK, NULL, SHAPE, NO, ALIGN, WS, DTYPE = (L.NF4_OK, L.NF4_ERR_NULL, L.NF4_ERR_SHAPE, L.NF4_ERR_UNSUPPORTED, L.NF4_ERR_ALIGN,
                                         L.NF4_ERR_WORKSPACE, L.NF4_ERR_DTYPE)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from nf4_bit_weight_amd import build as B
        B.build()
    return L.lib()


@pytest.mark.parametrize("header,count", [("nf4_experts.h", 8), ("nf4_int8.h", 5)])
def test_exports_every_declared_symbol(lib, header, count):
    text = open(os.path.join(ROOT, "include", header)).read()
    names = sorted(set(re.findall(r"\b(nf4_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S))))
    assert len(names) == count
    for n in names:
        assert hasattr(lib, n) and n in L.SIGNATURES, n
    for name, value in re.findall(r"#define\s+(NF4_[A-Z0-9_]+)\s+(\d+)", text):
        assert int(value) == getattr(L, name), name


def call(fn, base, order, **kw):
    a = dict(base, **kw)
    assert set(kw) <= set(base), kw
    return fn(*(a[n] for n in order.split()), None)


def test_route_refuses(lib):
    base = dict(l=A, dt=0, st=16, T=4, E=16, k=2, bias=A, score=0, g=4, tg=2, gs=0, re=1, scale=1.0, w=A, e=A, off=A, tok=A, slot=A,
                ws=A, wsb=1 << 20)

    def f(**kw):
        return call(lib.nf4_route_fwd, base, "l dt st T E k bias score g tg gs re scale w e off tok slot ws wsb", **kw)
    assert f(l=None) == f(w=None) == f(e=None) == f(off=None) == f(tok=None) == f(slot=None) == NULL
    assert f(T=-1) == f(E=0) == f(k=0) == f(k=17) == f(st=-1) == f(g=0) == f(g=3) == f(tg=0) == f(tg=5) == SHAPE
    for s in (0.0, -1.0, math.inf, math.nan):
        assert f(scale=s) == SHAPE
    assert f(E=1025) == f(E=512, k=65, g=1, tg=1) == f(T=1 << 30) == f(T=1 << 26, k=1) == f(score=2) == f(gs=2) == NO
    assert f(dt=2) == DTYPE
    assert f(l=A + 2) == f(bias=A + 2) == f(w=A + 1) == f(slot=A + 2) == f(T=4000, ws=BAD) == ALIGN
    assert lib.nf4_expert_plan_workspace(4, 2, 16) == 0                     # one workgroup does it all
    need = lib.nf4_expert_plan_workspace(4000, 2, 16)
    assert 0 < need < BIG
    assert f(T=4000, ws=None) == f(T=4000, wsb=need - 1) == WS
    assert lib.nf4_expert_plan_workspace(-1, 2, 16) == lib.nf4_expert_plan_workspace(4, 0, 16) == lib.nf4_expert_plan_workspace(4, 2, 0) == BIG
    # without a plan, and without tokens
    assert f(T=0, l=None, w=None, e=None, off=None, tok=None, slot=None, ws=None, wsb=0) == OK


def test_route_bwd_refuses(lib):
    base = dict(g=A, l=A, dt=1, st=16, T=4, E=16, k=2, w=A, e=A, score=1, re=0, scale=1.0, out=A)

    def f(**kw):
        return call(lib.nf4_route_bwd, base, "g l dt st T E k w e score re scale out", **kw)
    assert f(g=None) == f(l=None) == f(w=None) == f(e=None) == f(out=None) == NULL
    assert f(T=-1) == f(k=17) == f(st=-16) == f(scale=0.0) == SHAPE
    assert f(E=2000) == f(score=7) == NO
    assert f(dt=5) == DTYPE
    assert f(out=A + 1) == f(g=A + 2) == ALIGN
    assert f(T=0, g=None, l=None, w=None, e=None, out=None) == OK


def test_plan_refuses(lib):
    base = dict(e=A, T=4, k=2, E=16, off=A, tok=A, slot=A, ws=A, wsb=1 << 20)

    def f(**kw):
        return call(lib.nf4_expert_plan, base, "e T k E off tok slot ws wsb", **kw)
    assert f(e=None) == f(off=None) == f(tok=None) == f(slot=None) == NULL
    assert f(T=-1) == f(k=0) == f(E=0) == SHAPE
    assert f(k=65) == f(E=1025) == f(T=1 << 30) == NO
    assert f(e=A + 2) == f(T=4000, ws=BAD) == ALIGN
    assert f(T=4000, ws=None) == f(T=4000, wsb=16) == WS


def test_rows_refuse(lib):
    def gather(x=A, dt=0, st=64, T=4, H=64, k=2, slots=A, end=A, rows=A, fill=1):
        return lib.nf4_expert_gather(x, dt, st, T, H, k, slots, end, rows, fill, None)

    def gather_bwd(g=A, dt=0, T=4, H=64, k=2, slots=A, out=A):
        return lib.nf4_expert_gather_bwd(g, dt, T, H, k, slots, out, None)

    def combine(rows=A, dt=0, T=4, H=64, k=2, w=A, slots=A, out=A):
        return lib.nf4_expert_combine_fwd(rows, dt, T, H, k, w, slots, out, None)

    def combine_bwd(g=A, st=64, rows=A, dt=0, T=4, H=64, k=2, w=A, slots=A, end=A, gr=A, gw=A, fill=1):
        return lib.nf4_expert_combine_bwd(g, st, rows, dt, T, H, k, w, slots, end, gr, gw, fill, None)
    for f in (gather, gather_bwd, combine, combine_bwd):
        assert f(dt=2) == DTYPE
        assert f(T=-1) == f(H=-1) == f(k=0) == SHAPE
        assert f(k=65) == f(T=1 << 29) == f(T=1 << 24) == f(H=(1 << 24) + 1) == NO
        assert f(slots=None) == NULL
        assert f(slots=A + 2) == ALIGN
    assert gather(x=None) == gather(rows=None) == gather(end=None) == NULL
    assert gather(st=-1) == combine_bwd(st=-1) == SHAPE
    assert gather(x=A + 2) == gather_bwd(g=A + 2) == combine(w=A + 2) == combine_bwd(gw=A + 2) == ALIGN
    assert gather_bwd(g=None) == gather_bwd(out=None) == combine(rows=None) == combine(w=None) == combine(out=None) == NULL
    assert combine_bwd(g=None) == combine_bwd(rows=None) == combine_bwd(w=None) == combine_bwd(end=None) == NULL
    assert combine_bwd(gr=None, gw=None) == gather(T=0, x=None, rows=None) == gather(H=0, x=None, rows=None) == OK
    assert combine(T=0, rows=None, w=None, slots=None, out=None) == gather_bwd(T=0, g=None, slots=None, out=None) == OK


def test_rows_refuse_what_no_launch_holds(lib):
    """A launch has at most 65535 workgroups across a row and 2^32 threads, also of rows without elements."""
    assert lib.nf4_expert_gather(A, 0, 64, 4, (1 << 23) + 1, 2, A, A, A, 1, None) == NO
    assert lib.nf4_expert_combine_fwd(A, 0, 4, 65536 * 256, 2, A, A, A, None) == NO
    assert lib.nf4_expert_combine_bwd(None, 0, None, 0, 1 << 24, 0, 1, A, A, A, A, A, 1, None) == NO


def test_int8_refuses(lib):
    base = dict(x=A, dt=1, st=256, xs=None, M=4, q=A, s=A, N=32, K=256, bias=None, y=A, yd=0, ws=A, wsb=1 << 30)

    def f(**kw):
        return call(lib.nf4_int8_matmul, base, "x dt st xs M q s N K bias y yd ws wsb", **kw)
    g_base = dict(x=A, dt=1, st=256, xs=None, rows=4, tok=A, off=A, E=2, M=8, q=A, s=A, N=32, K=256, y=A, yd=0, fill=1, ws=A, wsb=1 << 30)

    def g(**kw):
        return call(lib.nf4_int8_grouped_matmul, g_base, "x dt st xs rows tok off E M q s N K y yd fill ws wsb", **kw)
    for h in (f, g):
        assert h(x=None) == h(q=None) == h(s=None) == h(y=None) == h(dt=2) == NULL     # integers without their scales
        assert h(M=-1) == h(N=-1) == h(K=-1) == h(st=-1) == SHAPE
        assert h(K=130945) == h(M=(1 << 28) + 1) == h(N=(1 << 28) + 1) == NO
        assert h(dt=3) == h(yd=2) == DTYPE
        assert h(q=BAD) == h(y=BAD) == h(ws=BAD) == h(x=A + 1) == h(dt=2, x=BAD, xs=A) == ALIGN
        assert h(ws=None) == h(wsb=256) == WS
        assert h(M=0, x=None, q=None, s=None, y=None, **({"rows": 0} if h is g else {})) == OK
        assert h(N=0, q=None, s=None, y=None) == OK
    assert g(E=0) == g(rows=3, tok=None) == g(rows=0, x=None) == SHAPE
    assert g(off=None) == NULL
    assert g(E=1025) == NO
    assert g(off=A + 2) == g(tok=A + 2) == ALIGN
    assert [lib.nf4_int8_row_bytes(k) for k in (-1, 0, 1, 128, 129)] == [-1, 0, 128, 128, 256]
    assert lib.nf4_int8_workspace(1, -1, 4, 32, 256, 0) == BIG and lib.nf4_int8_workspace(5, 4, 4, 32, 256, 0) == BIG
    assert lib.nf4_int8_workspace(1, 4, 4, 32, 256, 0) >= 4 * 256 + 16

    def quantize(x=A, dt=0, st=8, M=2, K=8, q=A, s=A):
        return lib.nf4_int8_quantize(x, dt, st, M, K, q, s, None)
    assert quantize(x=None) == quantize(q=None) == quantize(s=None) == NULL
    assert quantize(M=-1) == quantize(K=-1) == quantize(st=-1) == SHAPE
    assert quantize(K=130945) == quantize(M=1 << 24) == NO
    assert quantize(dt=2) == DTYPE
    assert quantize(q=BAD) == quantize(x=A + 2) == ALIGN
    assert quantize(M=0, x=None, q=None, s=None) == OK


def test_python_refuses_host_tensors():
    i = torch.zeros((2, 1), dtype=torch.int32)
    r = NF4Routing(torch.zeros(2, 1), i, torch.zeros(3, dtype=torch.int32), i.flatten(), i)
    assert (r.num_experts, r.top_k) == (2, 1)
    x = torch.zeros((2, 16))
    w = NF4Int8(torch.zeros((4, 128), dtype=torch.int8), torch.zeros(4), 4, 16)
    assert w.nbytes() == 4 * 132 and w.per_expert(2).N == 2
    with pytest.raises(ValueError, match="do not split"):
        w.per_expert(3)
    for f in (lambda: nf4_route(x, 1), lambda: nf4_expert_gather(x, r), lambda: nf4_expert_combine(x, r), lambda: nf4_expert_plan(i, 2),
              lambda: nf4_int8_quantize(x), lambda: nf4_int8_matmul(x, w)):
        with pytest.raises(ValueError, match="device"):
            f()
    with pytest.raises(ValueError, match="score"):
        nf4_route(x, 1, score=["softmax"])


def test_plain_forms():
    """The oracles themselves, on cases that can be seen through."""
    l = torch.log(torch.tensor([[0.1, 0.4, 0.2, 0.3]]))
    w, e = R.route(l, 2)
    assert e.tolist() == [[1, 3]] and torch.allclose(w, torch.tensor([[0.4, 0.3]], dtype=torch.float64))
    w, e = R.route(l, 2, renormalize=True, scale=7.0)
    assert torch.allclose(w, torch.tensor([[4.0, 3.0]], dtype=torch.float64))
    assert R.choose(l[0].double().tolist(), 2, groups=2, top_groups=1, group_score="top2") in ([1, 0], [3, 2])    # 0.5 each, up to rounding
    assert R.choose([0.0, 5.0, 3.0, 3.0], 2, groups=2, top_groups=1, group_score="top2", score="sigmoid") == [2, 3]
    assert R.choose([0.0, 5.0, 3.0, 3.0], 2, groups=2, top_groups=1) == [1, 0]
    assert R.choose([0.0, 0.0, -math.inf], 3) == [0, 1, -1]
    assert R.choose([1.0, 0.0], 1, score="sigmoid", bias=[0.0, 0.5]) == [1]
    off, tok, slot = R.plan(torch.tensor([[1, 0], [1, -1], [2, 1]], dtype=torch.int32), 3)
    assert off.tolist() == [0, 1, 4, 5] and tok.tolist() == [0, 0, 1, 2, 2, -1] and slot.tolist() == [[1, 0], [2, -1], [4, 3]]
    q, s = R.quantize(torch.tensor([[127.0, 0.5, 1.5, -2.5, -126.6], [0.0, 0.0, 0.0, 0.0, 0.0]]))
    assert q.tolist() == [[127, 0, 2, -2, -127], [0] * 5] and s.tolist() == [1.0, 0.0]


@pytest.mark.parametrize("mistake", ["ties", "bias in the weight", "group sum", "order"])
def test_a_planted_mistake_is_seen(mistake):
    """Each plausible mistake in the choice changes an answer that the GPU tests compare."""
    l, bias = R.normal(1, 40, 16), 0.3 * R.normal(2, 16)
    l[0] = 0.0
    w, e = R.route(l, 4, score="sigmoid", bias=bias, groups=4, top_groups=2, group_score="top2")
    if mistake == "ties":
        other = R.route(l.flip(1), 4)[1]
        assert not torch.equal(15 - other, R.route(l, 4)[1])
    elif mistake == "bias in the weight":
        s = torch.sigmoid(l.double()) + bias.double()
        assert not torch.allclose(s.gather(1, e.long()), w)
    elif mistake == "group sum":
        assert not torch.equal(R.route(l, 4, score="sigmoid", bias=bias, groups=4, top_groups=2)[1], e)
    else:
        assert not torch.equal(R.route(l, 4, score="sigmoid", groups=4, top_groups=2, group_score="top2")[1], e)
