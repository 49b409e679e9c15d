"""Weights and gradients of rows masked with the type's lowest number, to bounds
that hold them there too (expert_room.py)."""

import pytest
import torch

import expert_ref as R
import expert_room as X
from nf4_bit_weight_amd import nf4_route, nf4_route_bwd

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.mark.parametrize("E", [6, 16, 60, 64, 200, 512, 1000])
@pytest.mark.parametrize("dtype", R.BOTH)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_masked_rows(E, dtype, score, renormalize):
    l = X.masked_rows(E, E, dtype)
    bias = 0.01 * R.normal(1, E)
    for how in (dict(), dict(bias=bias), dict(groups=2, top_groups=1, group_score="top2"), dict(groups=2, top_groups=2, bias=bias)):
        kw = dict(score=score, renormalize=renormalize, scale=1.5, **how)
        leaf = l.to(DEV).requires_grad_()
        r = nf4_route(leaf, 6 if "groups" not in how else 3, **{n: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for n, v in kw.items()})
        w, e = R.route(l, r.top_k, **kw)
        assert torch.equal(r.experts.cpu(), e), kw
        X.weights_within(r.weights, w, l, str(kw))
        g = R.normal(E + 1, *w.shape)
        got, = torch.autograd.grad(r.weights, leaf, g.to(DEV))
        X.gradient_within(got, g, l, r.weights.detach().cpu(), e, score, renormalize, 1.5, dtype)
        assert torch.equal(got, nf4_route_bwd(g.to(DEV), leaf.detach(), r, score=score, renormalize=renormalize, scale=1.5))


@pytest.mark.parametrize("T,E,k", [(70, 16, 5), (129, 64, 8), (23, 256, 8), (5, 512, 10), (3, 1024, 64)])
@pytest.mark.parametrize("dtype", R.BOTH)
def test_ordinary_rows(T, E, k, dtype):
    l = (2 * R.normal(T + E, T, E)).to(dtype)
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            r = nf4_route(l.to(DEV), k, score=score, renormalize=renormalize)
            X.weights_within(r.weights, R.route(l, k, score=score, renormalize=renormalize)[0], l)
