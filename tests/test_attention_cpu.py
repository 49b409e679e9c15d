"""Host-side checks of the attention operators' C ABI (nf4_attn.h): exports, and
what each call refuses.  No device work is issued: every call here fails its
checks or is empty."""

import ctypes
import os
import re

import pytest
import torch

import attn_ref as R
from nf4_bit_weight_amd import _lib as L
from nf4_bit_weight_amd import nf4_kv_append, nf4_kv_attention, nf4_kv_cache, nf4_prompt_attention

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nf4_attn.h")
A, BAD = 0x10000, 0x10008          # aligned and not; never dereferenced
BIG = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from nf4_bit_weight_amd import build as B
        B.build()
    return L.lib()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(nf4_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 7
    for n in names:
        assert hasattr(lib, n) and n in L.SIGNATURES, n


def append(lib, **kw):
    a = dict(q=A, qs=256, k=A, ks=128, v=A, vs=128, T=2, Hq=4, off=A, lens=A, B=1, table=A, width=1, inv=A, rotary=64,
             inter=0, kc=A, ksc=A, vc=A, vsc=A, P=1, page=16, Hkv=2, D=64, qo=A, ko=A, fill=1)
    a.update(kw)
    return lib.nf4_kv_append(*(a[n] for n in ("q", "qs", "k", "ks", "v", "vs", "T", "Hq", "off", "lens", "B", "table",
                                             "width", "inv", "rotary", "inter", "kc", "ksc", "vc", "vsc", "P", "page",
                                             "Hkv", "D", "qo", "ko", "fill")), None)


def attention(lib, **kw):
    a = dict(q=A, qs=256, T=2, Hq=4, off=A, lens=A, B=1, table=A, width=1, kc=A, ksc=A, vc=A, vsc=A, P=1, page=16, Hkv=2,
             D=64, scale=0.125, out=A, fill=1, ws=A, wsb=0)
    a.update(kw)
    return lib.nf4_kv_attention(*(a[n] for n in ("q", "qs", "T", "Hq", "off", "lens", "B", "table", "width", "kc", "ksc",
                                                "vc", "vsc", "P", "page", "Hkv", "D", "scale", "out", "fill", "ws",
                                                "wsb")), None)


COMMON = [
    (dict(T=-1), L.NF4_ERR_SHAPE), (dict(B=-1), L.NF4_ERR_SHAPE), (dict(Hq=3), L.NF4_ERR_SHAPE),
    (dict(Hkv=0), L.NF4_ERR_SHAPE), (dict(D=96), L.NF4_ERR_UNSUPPORTED), (dict(T=2 ** 31), L.NF4_ERR_UNSUPPORTED),
    (dict(Hq=2048, Hkv=2), L.NF4_ERR_UNSUPPORTED), (dict(page=24), L.NF4_ERR_UNSUPPORTED), (dict(page=0), L.NF4_ERR_SHAPE),
    (dict(P=-1), L.NF4_ERR_SHAPE), (dict(kc=None), L.NF4_ERR_NULL), (dict(vsc=None), L.NF4_ERR_NULL),
    (dict(kc=BAD), L.NF4_ERR_ALIGN), (dict(ksc=BAD), L.NF4_ERR_ALIGN), (dict(off=None), L.NF4_ERR_SHAPE),
    (dict(lens=None), L.NF4_ERR_NULL), (dict(table=None), L.NF4_ERR_NULL), (dict(width=-1), L.NF4_ERR_SHAPE),
    (dict(width=2 ** 30), L.NF4_ERR_UNSUPPORTED), (dict(q=BAD), L.NF4_ERR_ALIGN), (dict(qs=257), L.NF4_ERR_ALIGN),
    (dict(qs=-8), L.NF4_ERR_SHAPE), (dict(off=A + 2), L.NF4_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,want", COMMON)
def test_cache_calls_refuse(lib, kw, want):
    assert append(lib, **kw) == want
    assert attention(lib, **kw) == want


def test_append_refuses(lib):
    assert append(lib, k=None) == L.NF4_ERR_NULL
    assert append(lib, v=None) == L.NF4_ERR_NULL
    assert append(lib, qo=None) == L.NF4_ERR_NULL
    assert append(lib, q=None) == L.NF4_ERR_NULL
    assert append(lib, inv=None) == L.NF4_ERR_NULL
    assert append(lib, rotary=24) == L.NF4_ERR_UNSUPPORTED
    assert append(lib, rotary=80) == L.NF4_ERR_SHAPE
    assert append(lib, ko=BAD) == L.NF4_ERR_ALIGN
    assert append(lib, vs=132) == L.NF4_ERR_ALIGN
    assert append(lib, T=0, k=None, v=None, q=None, qo=None) == L.NF4_OK


def test_attention_refuses(lib):
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert attention(lib, scale=s) == L.NF4_ERR_SHAPE
    assert attention(lib, q=None) == L.NF4_ERR_NULL
    assert attention(lib, out=None) == L.NF4_ERR_NULL
    assert attention(lib, out=BAD) == L.NF4_ERR_ALIGN
    assert attention(lib, T=0, q=None, out=None, ws=None) == L.NF4_OK
    need = lib.nf4_kv_attention_workspace(2, 1, 4, 2, 64, 100, 16)
    assert 0 < need < BIG
    assert attention(lib, width=100, wsb=need - 1) == L.NF4_ERR_WORKSPACE
    assert attention(lib, width=100, ws=None, wsb=need) == L.NF4_ERR_WORKSPACE
    assert attention(lib, width=100, ws=BAD, wsb=need) == L.NF4_ERR_ALIGN
    assert lib.nf4_kv_attention_workspace(2, 1, 4, 2, 64, 32, 16) == 0       # at most 512 tokens: nothing to join
    # more 128-token steps over all units than 32 bits count
    assert attention(lib, T=1 << 26, B=1 << 26, off=None, Hq=32, Hkv=32, D=64, width=1 << 16, page=256, P=1) == L.NF4_ERR_UNSUPPORTED
    assert lib.nf4_kv_attention_workspace(2, 1, 4, 3, 64, 1, 16) == BIG
    assert lib.nf4_kv_attention_workspace(0, 0, 4, 2, 64, 1, 16) == 0


def test_dequantize_refuses(lib):
    def f(T=2, off=A, lens=A, B=1, table=A, width=1, kc=A, P=1, page=16, H=2, D=64, ko=A, vo=A):
        return lib.nf4_kv_dequantize(T, off, lens, B, table, width, kc, A, A, A, P, page, H, D, ko, vo, 1, None)
    assert f(ko=None) == f(vo=None) == f(kc=None) == f(lens=None) == L.NF4_ERR_NULL
    assert f(off=None) == f(T=-1) == L.NF4_ERR_SHAPE
    assert f(D=80) == f(page=8) == L.NF4_ERR_UNSUPPORTED
    assert f(vo=BAD) == L.NF4_ERR_ALIGN
    assert f(T=0, ko=None, vo=None) == L.NF4_OK


def test_prompt_refuses(lib):
    def fwd(q=A, qs=256, k=A, ks=128, v=A, vs=128, T=4, off=A, B=1, Hq=4, Hkv=2, D=64, scale=0.125, out=A, lse=A):
        return lib.nf4_prompt_attention_fwd(q, qs, k, ks, v, vs, T, off, B, Hq, Hkv, D, scale, out, None, lse, 1, None)

    def bwd(g=A, gs=256, q=A, k=A, v=A, out=A, lse=A, T=4, off=A, B=1, Hq=4, Hkv=2, D=64, scale=0.125, gq=A, gk=A, gv=A,
            ws=A, wsb=1 << 30):
        return lib.nf4_prompt_attention_bwd(g, gs, q, 256, k, 128, v, 128, out, None, lse, T, off, B, Hq, Hkv, D, scale, gq, gk,
                                            gv, 1, ws, wsb, None)
    assert fwd(q=None) == fwd(k=None) == fwd(v=None) == fwd(off=None) == fwd(out=None) == L.NF4_ERR_NULL
    assert fwd(Hq=3) == fwd(T=-1) == fwd(ks=-8) == fwd(scale=0.0) == L.NF4_ERR_SHAPE
    assert fwd(D=32) == fwd(T=2 ** 31 - 1) == L.NF4_ERR_UNSUPPORTED
    assert fwd(B=2 ** 29 - 1, Hq=32, Hkv=32) == L.NF4_ERR_UNSUPPORTED      # more workgroups than a launch takes
    assert fwd(q=BAD) == fwd(ks=100) == fwd(out=BAD) == fwd(lse=A + 2) == L.NF4_ERR_ALIGN
    assert fwd(T=0, q=None, k=None, v=None, out=None, lse=None) == L.NF4_OK
    assert bwd(g=None) == bwd(out=None) == bwd(lse=None) == bwd(gq=None) == bwd(gk=None) == bwd(gv=None) == L.NF4_ERR_NULL
    assert bwd(gs=4) == bwd(gk=BAD) == bwd(ws=BAD) == L.NF4_ERR_ALIGN
    assert bwd(ws=None) == bwd(wsb=lib.nf4_prompt_attention_bwd_workspace(4, 1, 4, 2, 64) - 1) == L.NF4_ERR_WORKSPACE
    assert bwd(T=0, g=None, q=None, k=None, v=None, out=None, lse=None, gq=None, gk=None, gv=None, ws=None) == L.NF4_OK
    assert lib.nf4_prompt_attention_bwd_workspace(-1, 1, 4, 2, 64) == BIG


def test_python_refuses_host_tensors():
    cache = nf4_kv_cache(1, 1, 16, 64, device="cpu")
    assert (cache.pages, cache.kv_heads, cache.page_size, cache.head_dim) == (1, 1, 16, 64)
    assert cache.nbytes() == 16 * 2 * (32 + 4)
    x = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        nf4_kv_append(cache, x, x, i, i[None])
    with pytest.raises(ValueError, match="device"):
        nf4_kv_attention(x, cache, i, i[None])
    with pytest.raises(ValueError, match="device"):
        nf4_prompt_attention(x, x, x, i)
    for args in ((1, 1, 24, 64), (1, 1, 16, 96), (-1, 1, 16, 64), (1, 0, 16, 64)):
        with pytest.raises(ValueError):
            nf4_kv_cache(*args, device="cpu")


def test_reference_encoding_round_trip():
    """The oracle itself: a level times a scale comes back as itself, a random
    block within half of the widest step (1 of 6)."""
    lev = torch.cat((R.LEVELS, -R.LEVELS)).float().repeat(4)
    x = (lev * 0.75).to(torch.bfloat16)[None]
    c, s = R.encode(x)
    assert torch.equal(R.decode(c, s).float(), x.float())
    y = R.normal(1, 50, 128)
    c, s = R.encode(y)
    top = y.double().unflatten(-1, (-1, 64)).abs().amax(-1, keepdim=True)
    # half of the widest step, and the fp32 rounding of the scale
    assert ((R.decode(c, s) - y.double()).unflatten(-1, (-1, 64)).abs() <= top * (1 / 6 + 2.0 ** -20)).all()


def test_refuses_what_a_launch_cannot_take(lib):
    """Launches of 2^32 threads and (row, head) pairs beyond 32 bits are refused
    before anything is enqueued."""
    no = L.NF4_ERR_UNSUPPORTED
    assert append(lib, T=1 << 26) == no
    assert lib.nf4_kv_dequantize(1 << 26, A, A, 1, A, 1, A, A, A, A, 1, 16, 2, 64, A, A, 1, None) == no
    assert attention(lib, T=1 << 23, B=1 << 23, off=None, Hq=1024, Hkv=1) == no            # 2^33 pairs
    assert attention(lib, T=1 << 25, Hq=16, Hkv=16, width=4) == no                         # 2^24 units of 32 rows, whole
    assert attention(lib, T=1 << 22, Hq=16, Hkv=2, width=100, wsb=1 << 40) == no           # 2^24 groups of 4 in the join
    x = (A, 1024, A, 1024, A, 1024)

    def fwd(T, B, H):
        return lib.nf4_prompt_attention_fwd(*x, T, A, B, H, H, 64, 0.125, A, None, A, 1, None)

    def bwd(T, B, H):
        return lib.nf4_prompt_attention_bwd(A, 1024, *x, A, None, A, T, A, B, H, H, 64, 0.125, A, A, A, 1, A, 1 << 50, None)
    assert fwd(128, (1 << 20) - 1, 16) == no and bwd(128, (1 << 19) - 1, 16) == no
    assert fwd(1 << 28, 1, 16) == no and bwd(1 << 28, 1, 16) == no
