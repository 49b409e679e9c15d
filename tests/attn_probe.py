"""A cache in which every token can be seen: a query row picks one token and a
reference token with equal, dominating scores, so its output is the mean of
their values.  Without the token it is the reference's value, with the token
counted twice two thirds of the token's: both far outside what rounding does,
where a token among thousands of equal weight would hide in it.

Keys are zeros but for the picked tokens, which hold 6 in a direction of their
own, and the reference, which holds 6 in the last direction; values are +-6: all
kept exactly by the 4-bit encoding."""

import torch

TOP = 6.0
PICK = 5.0                         # query: a score of 5 * 6 = 30; n tokens of score 0 weigh n e^-30
# The two weights are equal and are rounded once to bf16 each (2^-8 of 3), the
# mean once (2^-8 of 6); 2^-8 more for the sums' 2^-20 and the others' n e^-30
# below 2^-13 for any n here.
ROOM = (3 + 3 + 6 + 1) * 2.0 ** -8


def values(n, heads, D, seed):
    g = torch.Generator().manual_seed(seed)
    return (TOP * (2 * torch.randint(0, 2, (n, heads, D), generator=g) - 1)).to(torch.bfloat16)


def keys(n, heads, D, picked, ref):
    k = torch.zeros((n, heads, D), dtype=torch.bfloat16)
    for j, p in enumerate(picked):
        k[p, :, j] = TOP
    k[ref, :, D - 1] = TOP
    return k


def query(D, j):
    q = torch.zeros(D, dtype=torch.bfloat16)
    q[j] = q[D - 1] = PICK
    return q


def wanted(v, p, ref):
    """[heads, D] of the row that picks token p."""
    return (v[p].double() + v[ref].double()) / 2
