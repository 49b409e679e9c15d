"""The workspace queries of nf4_attn.h and the calls that take the workspace
refuse the same sizes (host side, no device work)."""

import ctypes
import os

import pytest

from nf4_bit_weight_amd import _lib as L
from nf4_bit_weight_amd import nf4_kv_attention_workspace

BIG = ctypes.c_size_t(-1).value
A = 0x10000                        # aligned, never dereferenced: every call here is refused


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from nf4_bit_weight_amd import build as B
        B.build()
    return L.lib()


GOOD = dict(T=2, B=1, Hq=4, Hkv=2, D=64, width=100, page=16)
REFUSED = [
    dict(T=-1), dict(B=-1), dict(Hq=3), dict(Hkv=0), dict(D=96), dict(Hq=2048), dict(T=2 ** 31), dict(width=-1),
    dict(page=0), dict(page=-16), dict(page=8), dict(page=24),
    dict(width=2 ** 27), dict(width=2 ** 30),                                      # positions beyond 32 bits
    dict(T=1 << 20, B=1 << 20, Hq=32, Hkv=32, width=1 << 16, page=256),            # steps beyond 32 bits
    dict(T=1 << 23, B=1 << 23, Hq=1024, Hkv=1),                                    # (row, head) pairs beyond 32 bits
    dict(T=1 << 25, Hq=16, Hkv=16, width=4),                                       # whole units beyond a launch
    dict(T=1 << 22, Hq=16, Hkv=2),                                                 # the join beyond a launch
]


@pytest.mark.parametrize("change", REFUSED)
def test_cache_attention(lib, change):
    s = dict(GOOD, **change)
    sizes = [s[n] for n in ("T", "B", "Hq", "Hkv", "D", "width", "page")]
    status = lib.nf4_kv_attention(A, 256, s["T"], s["Hq"], A, A, s["B"], A, s["width"], A, A, A, A, 1, s["page"], s["Hkv"],
                                  s["D"], 0.125, A, 1, A, 1 << 50, None)
    assert status in (L.NF4_ERR_SHAPE, L.NF4_ERR_UNSUPPORTED)
    assert lib.nf4_kv_attention_workspace(*sizes) == BIG
    with pytest.raises(ValueError, match="unsupported"):
        nf4_kv_attention_workspace(*sizes)


def test_cache_attention_accepts(lib):
    assert 0 < lib.nf4_kv_attention_workspace(*GOOD.values()) < BIG
    assert lib.nf4_kv_attention_workspace(*dict(GOOD, T=0).values()) == 0
    assert lib.nf4_kv_attention_workspace(*dict(GOOD, width=0).values()) == 0


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(B=-1), dict(Hq=3), dict(D=32), dict(Hkv=0),
    dict(T=128, B=(1 << 19) - 1, Hq=16, Hkv=16), dict(T=1 << 28, Hq=16, Hkv=16), dict(T=1, B=8300, Hq=1024, Hkv=1024)])
def test_prompt_backward(lib, change):
    s = dict(dict(T=4, B=1, Hq=4, Hkv=2, D=64), **change)
    x = (A, 1024, A, 1024, A, 1024)
    status = lib.nf4_prompt_attention_bwd(A, 1024, *x, A, None, A, s["T"], A, s["B"], s["Hq"], s["Hkv"], s["D"], 0.125, A, A, A, 1,
                                          A, 1 << 50, None)
    assert status in (L.NF4_ERR_SHAPE, L.NF4_ERR_UNSUPPORTED)
    assert lib.nf4_prompt_attention_bwd_workspace(*s.values()) == BIG


def test_prompt_backward_accepts(lib):
    assert 0 < lib.nf4_prompt_attention_bwd_workspace(4, 1, 4, 2, 64) < BIG
    assert lib.nf4_prompt_attention_bwd_workspace(0, 1, 4, 2, 64) == 0
