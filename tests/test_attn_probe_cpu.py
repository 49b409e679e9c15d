"""The oracle of the visible-token probes, with mistakes planted in it."""

import pytest
import torch

import attn_probe as P
import attn_ref as R


@pytest.mark.parametrize("D", [64, 128])
def test_a_lost_or_doubled_token_shows(D):
    n, ref = 400, 250
    picked = list(range(100, 100 + D - 1))
    k, v = P.keys(n, 1, D, picked, ref), P.values(n, 1, D, 1)
    kd, vd = (R.decode(*R.encode(x)) for x in (k, v))
    assert torch.equal(kd, k.double()) and torch.equal(vd, v.double())
    for j in (0, 5, D - 2):
        q = P.query(D, j)[None, None].double()
        p = picked[j]
        want = P.wanted(v, p, ref)

        def off(order):
            seen = torch.ones(1, len(order), dtype=torch.bool)
            return float((R.attend(q, kd[order], vd[order], seen, 1.0)[0][0] - want).abs().max())
        everyone = list(range(n))
        assert off(everyone) <= P.ROOM / 100
        assert off([t for t in everyone if t != p]) > 10 * P.ROOM
        assert off([t for t in everyone if t != ref]) > 10 * P.ROOM
        assert off([*everyone, p]) > 10 * P.ROOM
        assert off([t for t in everyone if t // 128 != p // 128]) > 10 * P.ROOM
