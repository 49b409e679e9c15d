"""Calls at the edge of what the attention operators take: offsets that no call
should hold, the largest and smallest values, the paths of the launch rules
that ordinary sizes do not reach."""

import numpy as np
import pytest
import torch

import attn_ref as R
from nf4_bit_weight_amd import (nf4_kv_append, nf4_kv_attention, nf4_kv_cache, nf4_kv_dequantize)

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
