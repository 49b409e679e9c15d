"""The attention operators with the quantised projections around them, as a
model runs them: a prompt enters the cache and is answered, tokens follow one
by one, and a training step goes back through all of it."""

import numpy as np
import pytest
import torch

import attn_ref as R
import workloads as WL
from nf4_bit_weight_amd import (nf4_kv_append, nf4_kv_attention, nf4_kv_cache, nf4_linear, nf4_matmul_bwd_input,
                                nf4_matmul_fwd, nf4_prompt_attention, nf4_prompt_attention_bwd,
                                nf4_prompt_attention_fwd, nf4_quantize)

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
HID, HQ, HKV, D, PAGE = 256, 4, 2, 64, 16


def weights():
    code = torch.from_numpy(WL.nf4_code_np()).to(DEV)
    return [nf4_quantize(WL.gpu_weight_f32(n, k, seed=300 + i, device=DEV, std=0.06), code)
            for i, (n, k) in enumerate(((HQ * D, HID), (HKV * D, HID), (HKV * D, HID), (HID, HQ * D)))]


def freqs():
    return (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().to(DEV)


def test_prompt_then_tokens():
    wq, wk, wv, wo = weights()
    inv = freqs()
    prompt = [21, 50]
    B, steps, T = 2, 20, sum(prompt)
    cache = nf4_kv_cache(16, HKV, PAGE, D, DEV)
    table = torch.from_numpy(np.random.default_rng(1).permutation(16)[:10].reshape(2, 5).astype(np.int32)).to(DEV)
    lens = torch.tensor(prompt, dtype=torch.int32, device=DEV)
    off = R.offsets_of(prompt).to(DEV)
    kept = [[], []]                                            # (keys, values) of each sequence as the cache holds them

    def project(x):
        n = x.shape[0]
        return (nf4_matmul_fwd(x, wq).view(n, HQ, D), nf4_matmul_fwd(x, wk).view(n, HKV, D),
                nf4_matmul_fwd(x, wv).view(n, HKV, D))

    def keep(b, k, v):
        kept[b].append((R.decode(*R.encode(k)), R.decode(*R.encode(v))))

    x = R.normal(1, T, HID).to(DEV)
    q, k, v = project(x)
    qr, kr = nf4_kv_append(cache, k, v, lens, table, offsets=off, inv_freq=inv, q=q, return_k=True)
    y = nf4_prompt_attention(qr, kr, v, off)
    pos = torch.cat([torch.arange(n) for n in prompt])
    qh, kh = R.rotate(q.cpu(), pos, inv.cpu(), False), R.rotate(k.cpu(), pos, inv.cpu(), False)
    R.within(y, *R.prompt(qh, kh, v.cpu(), prompt, 0.125)["out"], "prompt")
    at = 0
    for b, n in enumerate(prompt):
        keep(b, kh[at:at + n], v.cpu()[at:at + n])
        at += n
    assert nf4_matmul_fwd(y.reshape(T, HQ * D), wo).shape == (T, HID)

    length = list(prompt)
    for i in range(steps):
        x = R.normal(50 + i, B, HID).to(DEV)
        q, k, v = project(x)
        lens += 1
        qr, _ = nf4_kv_append(cache, k, v, lens, table, inv_freq=inv, q=q)
        y = nf4_kv_attention(qr, cache, lens, table)
        for b in range(B):
            p = torch.tensor([length[b]])
            keep(b, R.rotate(k[b:b + 1].cpu(), p, inv.cpu(), False), v[b:b + 1].cpu())
            length[b] += 1
            kd, vd = (torch.cat([e[j] for e in kept[b]]) for j in (0, 1))
            want, bound = R.attend(R.rotate(q[b:b + 1].cpu(), p, inv.cpu(), False).double(), kd, vd,
                                   torch.ones(1, length[b], dtype=torch.bool), 0.125)
            R.within(y[b:b + 1], want, bound, f"step {i} sequence {b}")


def test_training_step_through_the_block():
    """The gradient of the block's input is the calls' own, one behind the other."""
    wq, wk, wv, wo = weights()
    lens = [33, 90]
    T, off = sum(lens), R.offsets_of(lens).to(DEV)
    x = R.normal(2, T, HID).to(DEV).requires_grad_()
    gy = R.normal(3, T, HID).to(DEV)
    q, k, v = (nf4_linear(x, w).view(T, -1, D) for w in (wq, wk, wv))
    y = nf4_linear(nf4_prompt_attention(q, k, v, off).reshape(T, HQ * D), wo)
    y.backward(gy)

    q2, k2, v2 = (nf4_matmul_fwd(x.detach(), w).view(T, -1, D) for w in (wq, wk, wv))
    out, rest, lse = nf4_prompt_attention_fwd(q2, k2, v2, off, for_backward=True)
    assert torch.equal(nf4_matmul_fwd(out.view(T, HQ * D), wo), y.detach())
    go = nf4_matmul_bwd_input(gy, wo).view(T, HQ, D)
    parts = [nf4_matmul_bwd_input(g.reshape(T, -1), w).double()
             for g, w in zip(nf4_prompt_attention_bwd(go, q2, k2, v2, out, rest, lse, off), (wq, wk, wv))]
    # the three come together in bf16: two roundings of sums of three terms
    room = 2 * R.U * sum(p.abs() for p in parts)
    assert ((x.grad.double() - sum(parts)).abs() <= room).all()
