"""The 4-bit paged cache on the GPU: append with rotation, read back, attention."""

import numpy as np
import pytest
import torch

import attn_ref as R
import workloads as WL
from nf4_bit_weight_amd import (NF4KVCache, api, nf4_kv_append, nf4_kv_attention, nf4_kv_attention_workspace,
                                nf4_kv_cache, nf4_kv_dequantize)

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def same_scale(a, b):
    return torch.equal(a.cpu().view(torch.int32), b.view(torch.int32)) or (
        torch.equal(torch.isnan(a.cpu()), torch.isnan(b)) and torch.equal(torch.nan_to_num(a.cpu()), torch.nan_to_num(b)))


def freqs(half):
    return (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()


def positions(lens, new):
    return torch.tensor([ln - n + j for ln, n in zip(lens, new) for j in range(n)], dtype=torch.int64)


def owners(new):
    return [b for b, n in enumerate(new) for _ in range(n)]


APPENDS = [
    # lens, new (None: one each), Hq, Hkv, D, page, rotary, interleaved
    ([1], None, 4, 1, 64, 16, 64, False),
    ([5, 17, 33, 1], None, 8, 2, 128, 16, 128, False),
    ([40, 0, 19, 64], [40, 0, 3, 1], 6, 2, 128, 48, 64, False),
    ([7, 300, 16], [7, 129, 16], 2, 2, 64, 32, 32, True),
    ([100000, 131071], [2, 5], 3, 1, 128, 256, 128, True),
    ([20, 20], [20, 20], 4, 4, 64, 16, 0, False),
    ([1100, 37], [1100, 37], 2, 1, 64, 64, 64, False),
    ([4100], [4100], 1, 1, 128, 16, 128, False),
]


@pytest.mark.parametrize("lens,new,Hq,Hkv,D,page,rotary,inter", APPENDS)
def test_append_bytes(lens, new, Hq, Hkv, D, page, rotary, inter):
    """Codes, scales and the rotated rows are the definition's, bit for bit, and
    the rest of the cache is left alone."""
    h = R.HostCache([max(n, 1) for n in lens], Hkv, page, D, seed=len(lens))
    cache, table = h.to(DEV)
    n = [1] * len(lens) if new is None else new
    T = sum(n)
    # slices of one joint projection
    joint = R.normal(3, T, Hq + 2 * Hkv, D)
    inv = freqs(rotary // 2) if rotary else None
    jd = joint.to(DEV)
    q, k, v = jd[:, :Hq], jd[:, Hq:Hq + Hkv], jd[:, Hq + Hkv:]
    qo, ko = nf4_kv_append(cache, k, v, i32(lens), table, offsets=None if new is None else R.offsets_of(n).to(DEV),
                           inv_freq=None if inv is None else inv.to(DEV), interleaved=inter, q=q, return_k=True)
    pos = positions(lens, n)
    qr, kr = (R.rotate(x, pos, inv, inter) for x in (joint[:, :Hq], joint[:, Hq:Hq + Hkv]))
    for t, (b, p) in enumerate(zip(owners(n), pos.tolist())):
        h.put(b, p, kr[t], joint[t, Hq + Hkv:])
    assert torch.equal(qo.cpu().view(torch.int16), qr.view(torch.int16))
    assert torch.equal(ko.cpu().view(torch.int16), kr.view(torch.int16))
    assert torch.equal(cache.k_codes.cpu(), h.k_codes) and torch.equal(cache.v_codes.cpu(), h.v_codes)
    assert same_scale(cache.k_scale, h.k_scale) and same_scale(cache.v_scale, h.v_scale)
    kd, vd = nf4_kv_dequantize(cache, i32(lens), table, offsets=None if new is None else R.offsets_of(n).to(DEV), rows=T)
    for t, (b, p) in enumerate(zip(owners(n), pos.tolist())):
        pg, i = int(h.table[b, p // page]), p % page
        for got, codes, scale in ((kd, h.k_codes, h.k_scale), (vd, h.v_codes, h.v_scale)):
            want = (R.decode(codes[pg, :, i], torch.ones_like(scale[pg, :, i])).float().unflatten(-1, (-1, 64))
                    * scale[pg, :, i][..., None]).flatten(-2).to(torch.bfloat16)
            assert torch.equal(got[t].cpu(), want)
        if t > 64:
            break


def test_append_without_queries_or_rotation():
    cache = nf4_kv_cache(2, 1, 16, 64, DEV)
    k, v = R.normal(1, 3, 1, 64), R.normal(2, 3, 1, 64)
    qo, ko = nf4_kv_append(cache, k.to(DEV), v.to(DEV), i32([3]), i32([[1]]), offsets=i32([0, 3]))
    assert qo is None and ko is None
    c, s = R.encode(k)
    assert torch.equal(cache.k_codes[1, 0, :3].cpu(), c[:, 0]) and torch.equal(cache.k_scale[1, 0, :3].cpu(), s[:, 0])
    assert not cache.k_codes[0].any() and not cache.k_codes[1, 0, 3:].any()


def test_special_blocks():
    """All-zero, tiny, huge, NaN and infinite blocks; every level and every
    half-way value."""
    rows = [torch.zeros(64), torch.full((64,), 2.0 ** -125), torch.full((64,), 3e38), torch.full((64,), 2.0 ** -120)]
    bad = R.normal(5, 64).float()
    bad[7] = float("nan")
    inf = R.normal(6, 64).float()
    inf[63] = -float("inf")
    ties = torch.zeros(64)
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    ties[:7] = torch.tensor(mids)
    ties[7:14] = -torch.tensor(mids)
    ties[14:22] = R.LEVELS.float()
    ties[22] = -0.0
    x = torch.stack([*rows, bad, inf, ties, ties * 2.0 ** 60, ties * 1.5]).to(torch.bfloat16)[:, None]
    T = x.shape[0]
    cache = nf4_kv_cache(1, 1, 16, 64, DEV)
    nf4_kv_append(cache, x.to(DEV), x.to(DEV), i32([T]), i32([[0]]), offsets=i32([0, T]))
    c, s = R.encode(x)
    assert torch.equal(cache.k_codes[0, 0, :T].cpu(), c[:, 0])
    assert torch.equal(cache.v_codes[0, 0, :T].cpu(), c[:, 0])
    assert same_scale(cache.k_scale[0, 0, :T], s[:, 0])
    kd, _ = nf4_kv_dequantize(cache, i32([T]), i32([[0]]), offsets=i32([0, T]), rows=T)
    got = kd[:, 0].cpu().float()
    assert torch.isnan(got[4]).all() and torch.isnan(got[5]).all() and not got[:2].any()
    # a block is at most half a level step off: 1 of 6 between the outermost levels
    fine = got[[0, 2, 3, 6, 7, 8]].double()
    assert ((fine - x[[0, 2, 3, 6, 7, 8], 0].double()).abs().amax(1) <= x[[0, 2, 3, 6, 7, 8], 0].double().abs().amax(1) * (1 / 6 + 2 ** -7)).all()


def test_levels_are_the_fp4_table():
    """The patterns' values are the framework's fp4 table times 6."""
    cache = nf4_kv_cache(1, 1, 16, 64, DEV)
    cache.k_codes[0, 0, 0, :8] = torch.arange(16, dtype=torch.uint8).view(8, 2).mul(torch.tensor([16, 1], dtype=torch.uint8)).sum(1).to(DEV)
    cache.k_scale[0, 0, 0] = 1.0
    kd, _ = nf4_kv_dequantize(cache, i32([1]), i32([[0]]))
    got = kd[0, 0, :16].double().cpu().numpy()
    assert np.allclose(np.sort(got), 6 * np.array(WL.FP4_LEVELS), atol=1e-12)


def test_holes_are_left_alone():
    """Positions below zero or behind the table, and pages outside the cache:
    nothing is written, the queries are rotated all the same, reads give zeros."""
    D, page, H = 64, 16, 2
    cache = nf4_kv_cache(3, H, page, D, DEV)
    table = i32([[0, 99, -5], [1, 2, -1], [2, 2, 2]])
    table[2] = -1
    lens, new = [40, 1, 60], [40, 3, 2]
    T = sum(new)
    k, v, q = R.normal(1, T, H, D), R.normal(2, T, H, D), R.normal(3, T, H, D)
    inv = freqs(D // 2)
    off = R.offsets_of(new).to(DEV)
    qo, _ = nf4_kv_append(cache, k.to(DEV), v.to(DEV), i32(lens), table, offsets=off, inv_freq=inv.to(DEV), q=q.to(DEV))
    pos = positions(lens, new)
    assert torch.equal(qo.cpu(), R.rotate(q, pos, inv, False))
    kr = R.rotate(k, pos, inv, False)
    c, s = R.encode(kr)
    assert torch.equal(cache.k_codes[0].cpu(), c[:16].transpose(0, 1))            # tokens 0..15 of the first sequence
    assert torch.equal(cache.k_codes[1, :, 0].cpu(), c[42])                       # token 0 of the second (rows -2, -1 are holes)
    assert not cache.k_codes[1, :, 1:].any() and not cache.k_codes[2].any()
    kd, vd = nf4_kv_dequantize(cache, i32(lens), table, offsets=off, rows=T)
    seen = torch.zeros(T, dtype=torch.bool)
    seen[:16] = True
    seen[42] = True
    assert not kd[~seen.to(DEV)].any() and not vd[~seen.to(DEV)].any()
    assert kd[seen.to(DEV)].any()


def test_rows_outside_sequences():
    """Rows behind the last sequence and before the first: zeros in a fresh
    result, as they were in one passed in; what they hold is never used."""
    D, H = 128, 1
    T, off = 9, i32([2, 4, 7])
    lens, table = i32([2, 3]), i32([[0], [1]])
    k = R.normal(1, T, H, D)
    k[7:] = float("nan")
    k[:2] = float("inf")
    kd = k.to(DEV)
    inside = torch.zeros(T, dtype=torch.bool, device=DEV)
    inside[2:7] = True

    def fresh():
        return nf4_kv_cache(2, H, 16, D, DEV)

    cache = fresh()
    qo, ko = nf4_kv_append(cache, kd, kd, lens, table, offsets=off, q=kd, return_k=True)
    assert torch.equal(qo[inside], kd[inside]) and not qo[~inside].any() and not ko[~inside].any()
    mark = torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device=DEV)
    q2, k2 = mark.clone(), mark.clone()
    nf4_kv_append(fresh(), kd, kd, lens, table, offsets=off, q=kd, q_out=q2, k_out=k2)
    for x in (q2, k2):
        assert torch.equal(x[inside], kd[inside]) and (x[~inside] == 3.0).all()
    a, b = nf4_kv_dequantize(cache, lens, table, offsets=off, rows=T)
    assert a[inside].any() and not a[~inside].any() and not b[~inside].any()
    a, b = nf4_kv_dequantize(cache, lens, table, offsets=off, rows=T, k_out=mark.clone(), v_out=mark.clone())
    assert (a[~inside] == 3.0).all() and (b[~inside] == 3.0).all()
    o = nf4_kv_attention(kd, cache, lens, table, offsets=off)
    assert torch.isfinite(o).all() and not o[~inside].any()
    o2 = nf4_kv_attention(kd, cache, lens, table, offsets=off, out=mark.clone())
    assert torch.equal(o2[inside], o[inside]) and (o2[~inside] == 3.0).all()


# ---- attention ---------------------------------------------------------------------

def check_attention(lens, new, Hq, Hkv, D, page, seed=0, width=None, scale=None, qscale=1.0):
    h = R.HostCache(lens, Hkv, page, D, seed=seed, width=width)
    h.fill(lens, 100 + seed)
    cache, table = h.to(DEV)
    n = [1] * len(lens) if new is None else new
    T = sum(n)
    q = R.normal(7 + seed, T, Hq, D, scale=qscale)
    off = None if new is None else R.offsets_of(n).to(DEV)
    out = nf4_kv_attention(q.to(DEV), cache, i32(lens), table, offsets=off, scale=scale)
    sc = D ** -0.5 if scale is None else scale
    want, bound, at = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64), 0
    for b, (ln, m) in enumerate(zip(lens, n)):
        k, v = h.dense(b, ln)
        pos = torch.arange(ln - m, ln)          # (rows before the first token see nothing)
        seen = torch.arange(ln)[None] <= pos[:, None]
        r = slice(at, at + m)
        want[r], bound[r] = R.attend(q[r].double(), k, v, seen, float(np.float32(sc)))
        at += m
    R.within(out, want, bound, f"{lens} {n} {Hq}/{Hkv} {D} {page}")
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 1), (10, 2), (17, 1)])
def test_attention_heads(D, Hq, Hkv):
    check_attention([37, 1, 130], None, Hq, Hkv, D, 16)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 257, 1000])
def test_attention_lengths(n):
    check_attention([n], None, 4, 2, 128, 48, seed=n)


@pytest.mark.parametrize("n", [1, 16, 129, 512, 513])
def test_attention_wide_tables(n):
    """Short sequences in a table for long ones, where workgroups share units."""
    check_attention([n, 0, 3], None, 4, 2, 64, 16, seed=n, width=200)


@pytest.mark.parametrize("page", [16, 32, 48, 80, 256])
def test_attention_pages(page):
    check_attention([page - 1, page, page + 1, 3 * page + 5], None, 4, 1, 64, page, seed=page)


@pytest.mark.parametrize("new", [[2, 0, 5], [9, 9, 9], [1, 33, 4], [16, 1, 40]])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_several_rows(new, D):
    check_attention([50, 200, 41], new, 10, 2, D, 16, seed=sum(new))


def test_attention_empty_rows_and_sequences():
    """Length 0, rows before the first token, a bad page inside a sequence."""
    D, page = 64, 16
    h = R.HostCache([40, 20], 1, page, D)
    h.fill([40, 20], 5)
    cache, table = h.to(DEV)
    table = torch.cat((table, table[:1]))
    lens, new = [40, 2, 0], [2, 4, 1]
    q = R.normal(9, 7, 2, D)
    out = nf4_kv_attention(q.to(DEV), cache, i32(lens), table, offsets=R.offsets_of(new).to(DEV))
    assert not out[2:4].any() and not out[6].any()              # rows -2, -1 of the second; the empty third
    assert out[4:6].any() and torch.isfinite(out).all()
    # tokens of a bad page are not seen
    t2 = table.clone()
    for bad in (-1, h.pages, 2 ** 31 - 1):
        t2[0, 1] = bad
        got = nf4_kv_attention(q[:1].to(DEV), cache, i32([40]), t2[:1])
        k, v = h.dense(0, 40)
        seen = torch.ones(1, 40, dtype=torch.bool)
        seen[:, 16:32] = False
        want, bound = R.attend(q[:1].double(), k, v, seen, float(np.float32(D ** -0.5)))
        R.within(got, want, bound, f"bad page {bad}")
    t2[0] = -1
    assert not nf4_kv_attention(q[:1].to(DEV), cache, i32([40]), t2[:1]).any()


def test_attention_length_beyond_table():
    """A length behind the table's end sees the tokens that the table holds."""
    D, page = 64, 16
    h = R.HostCache([32], 1, page, D)
    h.fill([32], 5)
    cache, table = h.to(DEV)
    q = R.normal(9, 1, 2, D).to(DEV)
    assert torch.equal(nf4_kv_attention(q, cache, i32([1000]), table), nf4_kv_attention(q, cache, i32([32]), table))
    empty = NF4KVCache(*(t[:0] for t in cache.tensors()))
    assert not nf4_kv_attention(q, empty, i32([32]), table).any()


def test_attention_nan_token_reaches_only_its_readers():
    D, page = 64, 16
    h = R.HostCache([20], 1, page, D)
    h.fill([20], 5)
    nan = torch.full((1, D), float("nan"), dtype=torch.bfloat16)
    h.put(0, 18, nan, nan)
    cache, table = h.to(DEV)
    out = nf4_kv_attention(R.normal(1, 4, 2, D).to(DEV), cache, i32([20]), table, offsets=i32([0, 4]))
    assert torch.isfinite(out[:2]).all() and torch.isnan(out[2:]).all()


def test_attention_many_sequences():
    """More sequences than a wave has lanes, shared unevenly among workers."""
    g = np.random.default_rng(3)
    lens = [int(x) for x in g.integers(0, 40, 150)]
    lens[77] = 2000
    h = R.HostCache(lens, 1, 16, 64)
    h.fill(lens, 11)
    cache, table = h.to(DEV)
    q = R.normal(5, 150, 4, 64)
    out = nf4_kv_attention(q.to(DEV), cache, i32(lens), table)
    for b, n in enumerate(lens):
        k, v = h.dense(b, n)
        want, bound = R.attend(q[b:b + 1].double(), k, v, torch.ones(1, n, dtype=torch.bool), 0.125)
        R.within(out[b:b + 1], want, bound, f"sequence {b} of {n}")


@pytest.mark.parametrize("count,longest,rows,Hq,Hkv,D", [
    (7, 700, 1, 4, 2, 128), (100, 1500, 1, 8, 8, 64), (40, 900, 5, 10, 2, 128), (300, 140, 2, 16, 8, 64)])
def test_attention_work_dealt_out(count, longest, rows, Hq, Hkv, D):
    """Fewer steps than workers, a few each and many each; sequences that one
    worker takes whole, ends in or begins in, and empty ones between them."""
    g = np.random.default_rng(count)
    lens = [int(x) for x in g.integers(1, longest + 1, count)]
    lens[2], lens[3], lens[count // 2] = 0, 1, longest
    new = [min(n, rows) for n in lens]
    check_attention(lens, new, Hq, Hkv, D, 16)


def test_attention_large_scores_and_scale():
    check_attention([300, 70], None, 4, 2, 128, 16, qscale=30.0)
    check_attention([300, 70], None, 4, 2, 128, 16, scale=0.01)


def test_attention_split_and_unsplit_agree():
    """One long sequence, split over workers and joined, against reading it back
    and computing densely in 64 bits on the device."""
    n, D, page, Hq, Hkv = 20011, 128, 64, 8, 2
    pages = -(-n // page)
    cache = nf4_kv_cache(pages, Hkv, page, D, DEV)
    table = i32(np.random.default_rng(1).permutation(pages)[None])
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn((n, Hkv, D), generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
    nf4_kv_append(cache, k, v, i32([n]), table, offsets=i32([0, n]))
    q = torch.randn((1, Hq, D), generator=g, device=DEV).to(torch.bfloat16)
    out = nf4_kv_attention(q, cache, i32([n]), table)
    codes = [R.encode(x.cpu()) for x in (k, v)]
    kd, vd = (R.decode(*c) for c in codes)
    want, bound = R.attend(q.cpu().double(), kd, vd, torch.ones(1, n, dtype=torch.bool), float(np.float32(D ** -0.5)))
    R.within(out, want, bound, "20011 tokens")
    for _ in range(3):
        assert torch.equal(nf4_kv_attention(q, cache, i32([n]), table), out)


def test_offsets_beyond_32_bits():
    """Pages whose bytes lie behind 2^32 in the codes and 2^31 elements in rows."""
    D, H, page = 128, 8, 128
    pages = 2 ** 32 // (H * page * D // 2) + 9
    cache = NF4KVCache(*(torch.empty((pages, H, page, n), dtype=t, device=DEV)
                         for n, t in ((64, torch.uint8), (2, torch.float32)) * 2))
    far = [pages - 1, 3, pages - 2]
    n = 2 * page + 5
    table = i32([far])
    k, v = R.normal(1, n, H, D), R.normal(2, n, H, D)
    nf4_kv_append(cache, k.to(DEV), v.to(DEV), i32([n]), table, offsets=i32([0, n]))
    kd, vd = nf4_kv_dequantize(cache, i32([n]), table, offsets=i32([0, n]), rows=n)
    ck, cv = R.encode(k), R.encode(v)
    assert torch.equal(cache.k_codes[far[2], :, :5].cpu(), ck[0][2 * page:].transpose(0, 1))
    q = R.normal(3, 1, H, D)
    out = nf4_kv_attention(q.to(DEV), cache, i32([n]), table)
    want, bound = R.attend(q.double(), R.decode(*ck), R.decode(*cv), torch.ones(1, n, dtype=torch.bool), float(np.float32(D ** -0.5)))
    R.within(out, want, bound, "far pages")


def test_repeatable_streams_and_workspaces():
    """The same bits on another stream, with a caller's workspace that holds
    anything, and from two calls in flight at once."""
    lens = [700, 3000, 1]
    h = R.HostCache(lens, 2, 32, 64)
    h.fill(lens, 3)
    cache, table = h.to(DEV)
    q = R.normal(2, 3, 8, 64).to(DEV)
    ln = i32(lens)
    ref = nf4_kv_attention(q, cache, ln, table)
    need = nf4_kv_attention_workspace(3, 3, 8, 2, 64, *table.shape[1:], 32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(nf4_kv_attention(q, cache, ln, table, ws=ws), ref)
    with pytest.raises(RuntimeError):
        nf4_kv_attention(q, cache, ln, table, ws=ws[:need - 16])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for s in (s1, s2):
        with torch.cuda.stream(s):
            outs += [nf4_kv_attention(q, cache, ln, table) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_decode_steps_in_a_graph():
    """Append and attention captured once and replayed as the sequences grow."""
    D, H, Hq, page, B = 64, 2, 4, 16, 3
    start = [5, 30, 47]
    steps = 20
    h = R.HostCache([n + steps for n in start], H, page, D)
    h.fill(start, 3)
    cache, table = h.to(DEV)
    eager, _ = h.to(DEV)
    lens = i32(start)
    inv = freqs(D // 2).to(DEV)
    q, k, v = (torch.zeros((B, n, D), dtype=torch.bfloat16, device=DEV) for n in (Hq, H, H))

    def step(c, lengths):
        qr, _ = nf4_kv_append(c, k, v, lengths, table, inv_freq=inv, q=q)
        return nf4_kv_attention(qr, c, lengths, table)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    scratch = NF4KVCache(*(t.clone() for t in cache.tensors()))
    with torch.cuda.stream(side):
        step(scratch, lens)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache, lens)
    for i in range(steps):
        for t, n, s in ((q, Hq, 1), (k, H, 2), (v, H, 3)):
            t.copy_(R.normal(1000 + 10 * i + s, B, n, D).to(DEV))
        lens += 1
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager, lens)
        assert torch.equal(out, want), i
        assert torch.equal(cache.k_codes, eager.k_codes)


def test_empty_calls():
    cache = nf4_kv_cache(1, 2, 16, 64, DEV)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    lens, table = i32([]), torch.empty((0, 1), dtype=torch.int32, device=DEV)
    api.nf4_reset_path_counts()
    q, k = nf4_kv_append(cache, none, none, lens, table, q=none, return_k=True)
    assert q.shape == k.shape == (0, 2, 64)
    assert nf4_kv_attention(none, cache, lens, table).shape == (0, 2, 64)
    assert nf4_kv_dequantize(cache, lens, table)[0].shape == (0, 2, 64)
    assert all(v == 0 for v in api.nf4_path_counts().values())


def test_path_counts():
    cache = nf4_kv_cache(1, 1, 16, 64, DEV)
    x = R.normal(1, 1, 1, 64).to(DEV)
    api.nf4_reset_path_counts()
    nf4_kv_append(cache, x, x, i32([1]), i32([[0]]))
    nf4_kv_dequantize(cache, i32([1]), i32([[0]]))
    nf4_kv_attention(x, cache, i32([1]), i32([[0]]))
    c = api.nf4_path_counts()
    assert (c["kv_append"], c["kv_dequantize"], c["kv_attention"]) == (1, 1, 1)


def test_refusals():
    cache = nf4_kv_cache(2, 2, 16, 64, DEV)
    x = R.normal(1, 3, 2, 64).to(DEV)
    lens, table, off = i32([3]), i32([[0]]), i32([0, 3])

    def bad(fn, *a, **kw):
        with pytest.raises(ValueError):
            fn(*a, **kw)

    bad(nf4_kv_attention, x, cache, lens, table)                                       # 3 rows, 1 sequence
    bad(nf4_kv_attention, x[:, :1], cache, lens, table, offsets=off)                   # 1 head on 2
    bad(nf4_kv_attention, x.float(), cache, lens, table, offsets=off)
    bad(nf4_kv_attention, x.transpose(0, 1), cache, lens, table, offsets=off)
    bad(nf4_kv_attention, x, cache, lens.long(), table, offsets=off)
    bad(nf4_kv_attention, x, cache, lens, table[0], offsets=off)
    bad(nf4_kv_attention, x, cache, lens, table, offsets=off[:1])
    bad(nf4_kv_attention, x, cache, lens, table, offsets=off, scale=0.0)
    bad(nf4_kv_attention, x, cache, lens, table, offsets=off, scale=float("nan"))
    bad(nf4_kv_attention, x, cache, lens, table, offsets=off, out=x[:, :1])
    bad(nf4_kv_attention, x.cpu(), cache, lens, table, offsets=off)
    bad(nf4_kv_append, cache, x, x[:2], lens, table, offsets=off)
    bad(nf4_kv_append, cache, x, x, lens, table, offsets=off, inv_freq=torch.ones(5, device=DEV))
    bad(nf4_kv_append, cache, x, x, lens, table, offsets=off, inv_freq=torch.ones(64, device=DEV))
    bad(nf4_kv_append, cache, x, x, lens, table, offsets=off, q=x, return_k=True, q_out=torch.empty_like(x))
    bad(nf4_kv_append, cache, x, x, lens, table, offsets=off, q_out=torch.empty_like(x))
    bad(nf4_kv_dequantize, cache, lens, table, offsets=off)
    bad(nf4_kv_dequantize, cache, lens, table, offsets=off, rows=3, k_out=torch.empty_like(x))
    bad(nf4_kv_cache, 1, 1, 24, 64, DEV)
    bad(nf4_kv_cache, 1, 1, 16, 96, DEV)
    odd = NF4KVCache(cache.k_codes, cache.k_scale[:1], cache.v_codes, cache.v_scale)
    bad(nf4_kv_attention, x, odd, lens, table, offsets=off)
    with pytest.raises(RuntimeError):                                                  # rows not 16-byte aligned
        y = torch.empty(3 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(3, 2, 64)
        nf4_kv_attention(y, cache, lens, table, offsets=off)


@pytest.mark.parametrize("width", [0, 2, 100])
def test_no_sequences(width):
    """Rows of a call without sequences are all padding: zeros in new results,
    left alone in given ones."""
    T, Hq, D = 5, 2, 64
    q, k = R.normal(7, T, Hq, D).to(DEV), R.normal(8, T, Hq, D).to(DEV)
    cache = nf4_kv_cache(3, Hq, 16, D, device=DEV)
    ln, off, table = i32([]), i32([0]), torch.zeros((0, width), dtype=torch.int32, device=DEV)
    assert not nf4_kv_attention(q, cache, ln, table, off).any()
    given = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
    nf4_kv_attention(q, cache, ln, table, off, out=given)
    assert (given == 3.0).all()
    qo, ko = nf4_kv_append(cache, k, k, ln, table, off, q=q, return_k=True)
    assert not qo.any() and not ko.any()
    assert not any(x.any() for x in nf4_kv_dequantize(cache, ln, table, off, rows=T))
    for n in (0, T):                                          # an empty first sequence, and none of the cache's pages
        empty = nf4_kv_attention(q, cache, i32([n]), torch.full((1, width), 9, dtype=torch.int32, device=DEV), i32([0, n]))
        assert not empty.any()
