"""Derivatives through the attention calls on the GPU: what they carry, and that
what they do not carry is refused rather than lost."""

import pytest
import torch
from torch.autograd import forward_ad

import attn_ref as R
from nf4_bit_weight_amd import nf4_prompt_attention

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def leaves(T, Hq, Hkv, D, seed=1):
    return [R.normal(seed + i, T, h, D).to(DEV).requires_grad_() for i, h in enumerate((Hq, Hkv, Hkv))]


def test_tangents_are_refused_in_both_directions():
    off = R.offsets_of([9]).to(DEV)
    xs = leaves(9, 2, 1, 64)
    out = nf4_prompt_attention(*xs, off)
    gy = R.normal(7, 9, 2, 64).to(DEV)
    with forward_ad.dual_level():
        for i in range(3):
            args = [x.detach() for x in xs]
            args[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(ValueError, match="tangent"):
                nf4_prompt_attention(*args, off)
        with pytest.raises(RuntimeError, match="tangent"):
            torch.autograd.grad(out, xs, forward_ad.make_dual(gy, gy), retain_graph=True)
    assert all(g.isfinite().all() for g in torch.autograd.grad(out, xs, gy))
