"""Calls at the edge of what the attention operators take: offsets that no call
should hold, the largest and smallest values, the paths of the launch rules
that ordinary sizes do not reach."""

import numpy as np
import pytest
import torch

import attn_ref as R
from nf4_bit_weight_amd import (nf4_kv_append, nf4_kv_attention, nf4_kv_cache, nf4_kv_dequantize, nf4_prompt_attention,
                                nf4_prompt_attention_fwd)

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def shuffled(lens, page, width=None, seed=1):
    """(page table [B, width], pages) of sequences of these lengths."""
    need = [-(-n // page) for n in lens]
    width = max(need) if width is None else width
    order = np.random.default_rng(seed).permutation(sum(need))
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return i32(table), sum(need)


@pytest.mark.parametrize("last", [0, -7, 6])
def test_decreasing_offsets(last):
    """A last offset before the others: which rows are found is not promised, but
    the calls end, read nothing out of range, and a row is right or zeros."""
    lens, T, Hq, Hkv, D, page = [4000, 300], 10, 8, 2, 128, 16
    table, pages = shuffled(lens, page)
    cache = nf4_kv_cache(pages, Hkv, page, D, DEV)
    k, v = (R.normal(s, sum(lens), Hkv, D).to(DEV) for s in (1, 2))
    nf4_kv_append(cache, k, v, i32(lens), table, R.offsets_of(lens).to(DEV))
    q = R.normal(3, T, Hq, D).to(DEV)

    def rows(off):
        return (nf4_kv_attention(q, cache, i32(lens), table, i32(off)),
                *nf4_kv_dequantize(cache, i32(lens), table, i32(off), rows=T))
    for got, right in zip(rows([5, 10, last]), rows([5, 10, 10])):
        for t in range(T):
            assert torch.equal(got[t], right[t]) or not got[t].any(), t
        assert right[5:].any() and not got[:5].any()


# ---- values at both ends of the range -----------------------------------------------
# 3e38 leaves room for the kernels' roundings below the largest bf16 (3.39e38),
# 2^-80 for sums of a few hundred weights above the smallest.

def rising(n, heads, D):
    """Keys whose scores with a query of ones at element 0 rise from 0 to 4.8:
    weights that grow by less than the running maximum's slack."""
    k = torch.zeros((n, heads, D), dtype=torch.bfloat16)
    k[:, :, 0] = (4.8 * torch.arange(n) / n).to(torch.bfloat16)[:, None]
    return k


def ends(n, heads, D, top, alike):
    v = torch.full((n, heads, D), top)
    if not alike:
        v *= torch.sign(torch.randn(v.shape, generator=torch.Generator().manual_seed(n)))
    return v.to(torch.bfloat16)


@pytest.mark.parametrize("top", [3e38, 2.0 ** -80])
@pytest.mark.parametrize("alike", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_values_at_the_ends(D, alike, top):
    lens, Hq, Hkv = [1, 2, 200, 130], 4, 2
    T = sum(lens)
    q = torch.zeros((T, Hq, D), dtype=torch.bfloat16)
    q[:, ::2, 0] = 1.0                                         # every other head weighs all keys alike
    k, v = torch.cat([rising(n, Hkv, D) for n in lens]), ends(T, Hkv, D, top, alike)
    out = nf4_prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), R.offsets_of(lens).to(DEV), 1.0)
    R.within(out, *R.prompt(q, k, v, lens, 1.0)["out"], f"values of {top}")


@pytest.mark.parametrize("top", [3e38, 2.0 ** -80])
@pytest.mark.parametrize("alike", [True, False])
@pytest.mark.parametrize("D,rows,lens", [(64, 1, [2, 300, 1]), (128, 1, [900, 2]), (64, 9, [400, 700]), (128, 9, [130, 1000])])
def test_cache_values_at_the_ends(D, rows, lens, alike, top):
    """In whole units and in ones that several workers share."""
    Hq, Hkv, page = 4, 2, 16
    new = [min(rows, n) for n in lens]
    h = R.HostCache(lens, Hkv, page, D, seed=3)
    for b, n in enumerate(lens):
        k, v = rising(n, Hkv, D), ends(n, Hkv, D, top, alike)
        for p in range(n):
            h.put(b, p, k[p], v[p])
    cache, table = h.to(DEV)
    q = torch.zeros((sum(new), Hq, D), dtype=torch.bfloat16)
    q[:, ::2, 0] = 1.0
    out = nf4_kv_attention(q.to(DEV), cache, i32(lens), table, R.offsets_of(new).to(DEV), 1.0)
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        kd, vd = h.dense(b, n)
        seen = torch.arange(n)[None] <= torch.arange(n - m, n)[:, None]
        want, bound = R.attend(q[at:at + m].double(), kd, vd, seen, 1.0)
        R.within(out[at:at + m], want, bound, f"values of {top}, sequence {b}")
        at += m


def test_flags_without_a_truth_value_are_refused():
    cache = nf4_kv_cache(1, 1, 16, 64, DEV)
    x = R.normal(1, 1, 1, 64).to(DEV)
    for name in ("interleaved", "return_k"):
        with pytest.raises(ValueError, match=name):
            nf4_kv_append(cache, x, x, i32([1]), i32([[0]]), **{name: np.ones(2)})
    with pytest.raises(ValueError, match="for_backward"):
        nf4_prompt_attention_fwd(x, x, x, i32([0, 1]), for_backward=np.ones(2))
