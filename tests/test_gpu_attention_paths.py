"""The paths of the attention operators' launch rules, each reached on purpose:
what the rule gives is computed here, so that a case that no longer reaches its
path fails instead of covering less."""

import numpy as np
import pytest
import torch

import attn_probe as P
import attn_ref as R
import test_gpu_kv_cache as KV
from nf4_bit_weight_amd import (nf4_kv_append, nf4_kv_attention, nf4_kv_attention_workspace, nf4_kv_cache, nf4_prompt_attention)

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


# ---- backward: the heads of a group over workgroups -----------------------------------

def head_parts(T, Hq, Hkv):
    cus = torch.cuda.get_device_properties(DEV).multi_processor_count
    return max(1, min(Hq // Hkv, cus // ((T // 128 + 1) * Hkv)))


def check_backward(lens, Hq, Hkv, D):
    T = sum(lens)
    q, gy = R.normal(21, T, Hq, D), R.normal(22, T, Hq, D)
    k, v = R.normal(23, T, Hkv, D), R.normal(24, T, Hkv, D)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    out = nf4_prompt_attention(*leaves, R.offsets_of(lens).to(DEV))
    grads = torch.autograd.grad(out, leaves, gy.to(DEV))
    want = R.prompt(q, k, v, lens, float(np.float32(D ** -0.5)), gy)
    for name, g in zip(("out", "grad_q", "grad_k", "grad_v"), (out, *grads)):
        R.within(g, *want[name], f"{lens} {Hq}/{Hkv} {D} {name}")
        # two roundings of at most 2^-8 each, of score gradients (or weights) and of the
        # result, without a common direction: in the norm no more than their sum
        e, (val, _) = g.detach().cpu().double() - want[name][0], want[name]
        assert float(e.norm()) <= 2.0 ** -7 * float(val.norm()), name


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,lens", [
    (64, 16, [500, 1, 300, 64, 235]),                          # several heads a workgroup, tiles of all kinds
    (32, 16, [128, 0, 700, 33, 190, 129]),
    (18, 18, [1000, 130]),                                     # one query head a key head, results straight to bf16
])
def test_backward_without_a_split(Hq, Hkv, lens, D):
    assert head_parts(sum(lens), Hq, Hkv) == 1
    check_backward(lens, Hq, Hkv, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,parts,lens", [(56, 8, 3, [600, 2, 300, 198]), (70, 10, 2, [64, 1000, 36])])
def test_backward_with_an_uneven_split(Hq, Hkv, parts, lens, D):
    assert head_parts(sum(lens), Hq, Hkv) == parts and Hq // Hkv % parts
    check_backward(lens, Hq, Hkv, D)


# ---- append: four rows a workgroup ------------------------------------------------------

@pytest.mark.parametrize("D,rotary,inter", [(64, 64, True), (64, 32, True), (64, 32, False), (64, 0, False),
                                            (128, 128, True), (128, 64, True), (128, 64, False), (128, 16, False)])
def test_append_four_rows(D, rotary, inter):
    lens, new = [1017, 300, 5], [1017, 9, 1]
    assert sum(new) >= 1024 and sum(new) % 4
    KV.test_append_bytes(lens, new, 3, 1, D, 48, rotary, inter)


# ---- cache attention: units shared by workers and joined --------------------------------

def plan(T, B, Hq, Hkv, D, width, page):
    """(row tiles of 16 a unit, whether a row's join takes a workgroup) of a call that shares its units."""
    assert nf4_kv_attention_workspace(T, B, Hq, Hkv, D, width, page) > 0, "whole units"
    return 1 if -(-T * (Hq // Hkv) // B) <= 16 else 2, T * Hq <= 1024


@pytest.mark.parametrize("tiles,wide,D,count,longest,rows,Hq,Hkv", [
    (1, True, 64, 7, 600, 1, 8, 2), (1, True, 128, 7, 600, 1, 8, 2),
    (1, False, 64, 64, 300, 1, 32, 8), (1, False, 128, 64, 300, 1, 32, 8), (1, False, 64, 300, 140, 2, 16, 8),
    (2, True, 64, 5, 500, 5, 16, 2), (2, True, 128, 5, 500, 5, 16, 2),
    (2, False, 64, 40, 300, 5, 16, 2), (2, False, 128, 40, 300, 5, 16, 2)])
def test_shared_units(tiles, wide, D, count, longest, rows, Hq, Hkv):
    g = np.random.default_rng(count + D)
    lens = [int(x) for x in g.integers(1, longest + 1, count)]
    lens[0], lens[-1], lens[count // 2] = 0, longest, 1
    new = [min(n, rows) for n in lens]
    width = 100
    assert plan(sum(new), count, Hq, Hkv, D, width, 16) == (tiles, wide)
    KV.check_attention(lens, new, Hq, Hkv, D, 16, seed=count, width=width)


def check_probes(n, positions, D, G, B, Hkv, page):
    """Every token of `positions` is seen, once, by the rows that pick it: B
    sequences over the same pages, one row of G heads on each key head."""
    Hq, pages = G * Hkv, -(-n // page)
    chunk = min(B * G, D - 1)
    table = np.random.default_rng(n).permutation(pages).astype(np.int32)
    lens, tables, off = i32([n] * B), i32(np.tile(table, (B, 1))), R.offsets_of([n]).to(DEV)
    cache = nf4_kv_cache(pages, Hkv, page, D, DEV)
    v = P.values(n, Hkv, D, n + D)
    for at in range(0, len(positions), chunk):
        picked = positions[at:at + chunk]
        ref = next(t for t in (*positions[at + chunk:at + chunk + 1], *range(n)) if t not in picked)
        nf4_kv_append(cache, P.keys(n, Hkv, D, picked, ref).to(DEV), v.to(DEV), lens[:1], tables[:1], off)
        which = (torch.arange(B * G) % len(picked)).view(B, G)  # the direction of each sequence's heads
        rows = torch.stack([P.query(D, j) for j in range(len(picked))])[which]       # [B, G, D]
        q = rows[:, None].expand(B, Hkv, G, D).reshape(B, Hq, D).contiguous()
        out = nf4_kv_attention(q.to(DEV), cache, lens, tables, scale=1.0).cpu().double().view(B, Hkv, G, D)
        want = torch.stack([P.wanted(v, p, ref) for p in picked])[which]             # [B, G, Hkv, D]
        miss = (out.transpose(1, 2) - want).abs().amax((2, 3))                       # [B, G]
        assert float(miss.max()) <= P.ROOM, (ref, sorted({picked[j] for j in which[miss > P.ROOM].tolist()}))


@pytest.mark.parametrize("tiles,wide,D,G,B,Hkv,n,page", [
    (1, True, 64, 16, 3, 2, 1100, 80), (1, True, 128, 16, 7, 2, 1500, 48),
    (1, False, 64, 4, 140, 2, 700, 16), (1, False, 128, 4, 140, 2, 700, 256),
    (2, True, 64, 30, 2, 2, 1100, 16), (2, True, 128, 32, 3, 2, 1500, 48),
    (2, False, 64, 20, 30, 2, 700, 48), (2, False, 128, 20, 30, 2, 700, 64)])
def test_every_token_is_seen_once(tiles, wide, D, G, B, Hkv, n, page):
    assert plan(B, B, G * Hkv, Hkv, D, -(-n // page), page) == (tiles, wide)
    check_probes(n, list(range(n)), D, G, B, Hkv, page)


@pytest.mark.parametrize("D,G,Hkv", [(128, 8, 2), (64, 4, 1), (128, 24, 1)])
def test_every_step_of_a_long_sequence_is_seen_once(D, G, Hkv):
    """The first and last token of every step of 128 tokens, and the tile and
    page edges of some, where hundreds of workers share one unit."""
    n, page = 20011, 64
    edges = sorted({p for s in range(0, n, 128) for p in (s - 1, s)} | {p for s in range(1280, 1664, 16) for p in (s - 1, s)} | {n - 1})
    check_probes(n, [p for p in edges if 0 <= p < n], D, G, 8 if D == 128 else 15, Hkv, page)


@pytest.mark.parametrize("G,D,n,page", [(4, 128, 480, 48), (8, 64, 257, 16), (24, 128, 300, 16)])
def test_every_token_of_whole_units_is_seen_once(G, D, n, page):
    assert nf4_kv_attention_workspace(2, 2, G, 1, D, -(-n // page), page) == 0
    check_probes(n, list(range(n)), D, G, 2, 1, page)
