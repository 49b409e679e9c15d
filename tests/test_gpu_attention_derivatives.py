"""Derivatives through the attention calls on the GPU: what they carry, and that
what they do not carry is refused rather than lost."""

import pytest
import torch
from torch.autograd import forward_ad

import attn_ref as R
from nf4_bit_weight_amd import _lib as L
from nf4_bit_weight_amd import api, nf4_prompt_attention
from nf4_bit_weight_amd._lib import NF4Error

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


def many_sequences(B, heads=1024):
    """One row in the last of B sequences, so many that the launch counts."""
    x = R.normal(1, 1, heads, 64).to(DEV)
    off = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    off[-1] = 1
    return x, off


def test_errors_are_alike_with_and_without_gradients():
    """What the C call refuses is an NF4Error with its status on both paths."""
    x, off = many_sequences(16500)                             # 2^32 threads and more
    for make in (lambda t: t, lambda t: t.clone().requires_grad_()):
        with pytest.raises(NF4Error) as e:
            nf4_prompt_attention(make(x), make(x), make(x), off)
        assert e.value.status == L.NF4_ERR_UNSUPPORTED


def test_backward_errors_carry_their_status():
    """A saved tensor that a hook gives back misaligned is refused by the C call,
    on autograd's thread."""
    off = R.offsets_of([9]).to(DEV)

    def shifted(t):
        if t.dtype != torch.bfloat16:
            return t
        return torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape).copy_(t)
    xs = leaves(9, 2, 1, 64)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, shifted):
        out = nf4_prompt_attention(*xs, off)
    with pytest.raises(NF4Error) as e:
        torch.autograd.grad(out, xs, torch.ones_like(out))
    assert e.value.status == L.NF4_ERR_ALIGN and "nf4_prompt_attention_bwd" in str(e.value)


def test_sizes_that_only_the_backward_refuses_are_refused_at_once():
    """grad_k's workgroups are twice as large: a call that records gradients must
    not run forward into a backward pass that cannot start."""
    x, off = many_sequences(8300)
    api.nf4_reset_path_counts()
    with pytest.raises(NF4Error) as e:
        nf4_prompt_attention(x.clone().requires_grad_(), x, x, off)
    assert e.value.status == L.NF4_ERR_UNSUPPORTED and "nf4_prompt_attention_bwd" in str(e.value)
    assert api.nf4_path_counts()["prompt_fwd"] == 0


@pytest.mark.parametrize("grads", [False, True])
def test_rows_too_far_apart_for_the_kernels_are_copied(grads):
    """Any layout is taken: rows more than 2^24 elements apart as well."""
    off = R.offsets_of([2]).to(DEV)
    xs = [x.detach() for x in leaves(2, 2, 2, 64)]
    gy = R.normal(9, 2, 2, 64).to(DEV)

    def far(x):
        y = torch.empty(2 ** 24 + 8 + 128, dtype=x.dtype, device=DEV).as_strided((2, 2, 64), (2 ** 24 + 8, 64, 1))
        return y.copy_(x)
    want = nf4_prompt_attention(*xs, off)
    assert torch.equal(nf4_prompt_attention(*(far(x) for x in xs), off), want)
    if grads:
        near = [x.clone().requires_grad_() for x in xs]
        g = torch.autograd.grad(nf4_prompt_attention(*near, off), near, gy)
        apart = [far(x).requires_grad_() for x in xs]
        got = torch.autograd.grad(nf4_prompt_attention(*apart, off), apart, far(gy))
        assert all(torch.equal(a, b) for a, b in zip(got, g))
