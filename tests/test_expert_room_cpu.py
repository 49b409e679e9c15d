"""The bounds of the masked rows (expert_room.py) let no wrong weight or gradient pass."""

import pytest
import torch

import expert_ref as R
import expert_room as X

FORMS = [(s, r) for s in ("softmax", "sigmoid") for r in (False, True)]


@pytest.mark.parametrize("dtype", R.BOTH)
@pytest.mark.parametrize("score,renormalize", FORMS)
def test_the_right_weights_pass_and_wrong_ones_do_not(dtype, score, renormalize):
    l = X.masked_rows(1, 32, dtype)
    w, e = R.route(l, 6, score=score, renormalize=renormalize, scale=1.5)
    X.weights_within(w.float(), w, l)
    seen = 0
    for t in range(l.shape[0]):
        j = int(w[t].argmax())
        if float(w[t, j]) < 1e-30:
            continue
        seen += 1
        for wrong in (float(w[t, j]) * 1.0001, float(w[t, j]) * 0.9999, 1e6, 0.0):
            bad = w.float().clone()
            bad[t, j] = wrong
            with pytest.raises(AssertionError):
                X.weights_within(bad, w, l)
    assert seen >= 6
    with pytest.raises(AssertionError):                         # a weight where nobody is chosen
        X.weights_within(torch.where(e < 0, 1e-6, w).float(), w, l)


@pytest.mark.parametrize("dtype", R.BOTH)
@pytest.mark.parametrize("score,renormalize", FORMS)
def test_wrong_gradients_do_not_pass(dtype, score, renormalize):
    l = X.masked_rows(2, 32, dtype)
    w, e = R.route(l, 6, score=score, renormalize=renormalize, scale=1.5)
    w = w.float()
    g = R.normal(3, *w.shape)
    want, _ = R.route_grad(g, l, w, e, score, renormalize, 1.5)
    how = (g, l, w, e, score, renormalize, 1.5, dtype)
    X.gradient_within(want.to(dtype), *how)
    step = {torch.float32: 1e-3, torch.bfloat16: 2e-2}[dtype]   # above the result's own rounding
    seen = 0
    for t in range(l.shape[0]):
        i = int(want[t].abs().argmax())
        if float(want[t, i].abs()) < 1e-3:
            continue
        seen += 1
        for wrong in (float(want[t, i]) * (1 + step), -float(want[t, i]), 1e6):
            bad = want.to(dtype)
            bad[t, i] = wrong
            with pytest.raises(AssertionError):
                X.gradient_within(bad, *how)
    assert seen >= 4
