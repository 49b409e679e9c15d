"""What the attention calls do with derivatives that they do not carry: they
refuse them, before they look at devices, so the refusals are seen on the host."""

import pytest
import torch
from torch.autograd import forward_ad

from nf4_bit_weight_amd import (NF4KVCache, nf4_kv_append, nf4_kv_attention, nf4_kv_cache, nf4_kv_dequantize,
                                nf4_prompt_attention, nf4_prompt_attention_bwd, nf4_prompt_attention_fwd)

X = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
I = torch.zeros(1, dtype=torch.int32)
LSE = torch.zeros((1, 1))


def cache(scale=None):
    c = nf4_kv_cache(1, 1, 16, 64, device="cpu")
    return c if scale is None else NF4KVCache(c.k_codes, c.k_scale, c.v_codes, scale(c.v_scale))


def calls(make):
    """Every call with `make` put around one of its inputs, at each place."""
    x = make(X)
    yield lambda: nf4_prompt_attention(x, X, X, I)
    yield lambda: nf4_prompt_attention(X, x, X, I)
    yield lambda: nf4_prompt_attention(X, X, x, I)
    yield from cache_calls(make)


def cache_calls(make):
    x = make(X)
    yield lambda: nf4_kv_append(cache(), x, X, I, I[None])
    yield lambda: nf4_kv_append(cache(), X, x, I, I[None])
    yield lambda: nf4_kv_append(cache(), X, X, I, I[None], q=x)
    yield lambda: nf4_kv_append(cache(), X, X, I, I[None], inv_freq=make(torch.ones(8)))
    yield lambda: nf4_kv_attention(x, cache(), I, I[None])
    yield lambda: nf4_kv_attention(X, cache(make), I, I[None])
    yield lambda: nf4_kv_dequantize(cache(make), I, I[None])


def test_forward_mode_tangents_are_refused():
    """A Jacobian-vector product must not lose the attention without an error."""
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))
        d = dual(X)
        raw = [lambda a=a: nf4_prompt_attention_fwd(*a, I) for a in ((d, X, X), (X, d, X), (X, X, d))]
        raw += [lambda a=a: nf4_prompt_attention_bwd(*a, None, LSE, I)
                for a in ((d, X, X, X, X), (X, d, X, X, X), (X, X, d, X, X), (X, X, X, d, X))]
        for call in [*calls(dual), *raw]:
            with pytest.raises(ValueError, match="tangent"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):      # no_grad does not switch them off
                call()
        with pytest.raises(ValueError, match="device"):
            nf4_prompt_attention(X, X, X, I)


def test_cache_calls_refuse_to_cut_a_graph():
    """Rotation and cache have no gradient: while gradients are recorded, inputs
    that want one are refused, not returned without their history."""
    def leaf(t):
        return t.clone().requires_grad_()
    for call in cache_calls(leaf):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device"):           # nothing is recorded: an ordinary call
            call()
    for call in cache_calls(lambda t: (leaf(t) * 1.0)):                             # a result further down
        with pytest.raises(ValueError, match="gradient"):
            call()
    for call in cache_calls(lambda t: leaf(t).detach()):
        with pytest.raises(ValueError, match="device"):
            call()
