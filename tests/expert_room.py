"""How far the weights of a choice may be off, also in rows that hold the type's
lowest number (a usual mask).

A weight is a quotient of e^(l - top) and a sum of such terms.  A difference l - top
loses half a step of its size, which is a relative error of |l - top| 2^-24 in the
term, but only while the term is there at all: beyond 104 below the top e^x is zero
in fp32 (2^-150 and less, against a sum of at least 1).  expf and the division lose
two steps each, the sums at most 16 + 6 + 6 roundings; numerator and denominator
both.  What is lost below fp32's normal numbers is under 1e-38."""

import torch

import expert_ref as R

SPAN = 104.0


def room(logits):
    """Relative error of the weights of each row of logits: [T, 1]."""
    l = logits.double()
    finite = torch.isfinite(l)
    top = torch.where(finite, l, -torch.inf).amax(-1, keepdim=True)
    below = torch.where(finite, top - l, 0.0).clamp(max=SPAN)
    return (2 * below.amax(-1, keepdim=True) + 48) * R.U32


def weights_within(got, want, logits, what=""):
    R.within(got, want, room(logits) * want + 1e-38, what)


def gradient_within(got, grad, logits, weights, experts, score, renormalize, scale, dtype):
    """Against the formula on the weights that the call gave (their sum D has k terms of two roundings)."""
    want, size = R.route_grad(grad, logits, weights, experts, score, renormalize, scale)
    bound = (room(logits) + 2 * weights.shape[1] * R.U32) * size
    R.within(got, want, R.rounded(bound, want, dtype), f"{score} {renormalize}")


def masked_rows(seed, E, dtype):
    """Rows of every way in which a mask of the type's lowest number, or of -inf, leaves them."""
    lowest = torch.finfo(dtype).min
    l = R.normal(seed, 12, E).to(dtype)
    l[0] = lowest                                               # all of them: equal scores
    l[1, 3 % E] = lowest                                        # one
    l[2, ::2] = lowest
    l[3, 1:] = lowest                                           # all but one
    l[4, 5:] = lowest                                           # fewer left than are chosen
    l[5, ::2], l[5, 1::2] = lowest, -torch.inf
    l[6, 2:] = -torch.inf
    l[6, 0] = lowest
    l[7] *= 30                                                  # terms that come and go at fp32's end
    l[8] = l[8] * 2 - 300
    l[9, : E // 2] = lowest / 2
    l[10] = -torch.inf
    return l
