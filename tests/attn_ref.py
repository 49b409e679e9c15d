"""Plain 64-bit forms of the attention operators on the host, with bounds on
what the kernels' roundings may add.

Roundings of the kernels: every softmax weight (times the value's scale) once to
bf16, every score gradient once to bf16, every output once to bf16 (each at most
2^-8 of the value); sums of n terms in fp32 in any order, taken with four times
the textbook n * 2^-24 of the summed magnitudes; the exponential and its
argument with 2^-21 (|score| + 1)."""

import numpy as np
import torch

U = 2.0 ** -8
F = 2.0 ** -22
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


# ---- the 4-bit encoding ------------------------------------------------------

def encode(x):
    """x [..., D] bf16 -> codes u8 [..., D/2], scale f32 [..., D/64]."""
    b = x.double().unflatten(-1, (-1, 64))
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    top = torch.where(bad, 1.0, b.abs().amax(-1, keepdim=True))
    dead = top < 2.0 ** -120
    y = torch.where(bad | dead, 0.0, 6.0 * b / torch.where(dead, 1.0, top))
    mids = (LEVELS[1:] + LEVELS[:-1]) / 2
    code = (y.abs()[..., None] >= mids).sum(-1)
    code = torch.where(bad | dead, 0, code + 8 * torch.signbit(b).long()).flatten(-2)
    scale = torch.where(dead, 0.0, top).float() / 6.0
    scale = torch.where(bad, float("nan"), scale)[..., 0]
    return (code[..., 0::2] * 16 + code[..., 1::2]).to(torch.uint8), scale


def decode(codes, scale):
    """-> [..., D] fp64"""
    c = codes.long()
    nib = torch.stack((c // 16, c % 16), -1).flatten(-2)
    v = torch.where(nib >= 8, -LEVELS[nib % 8], LEVELS[nib % 8])
    return (v.unflatten(-1, (-1, 64)) * scale.double()[..., None]).flatten(-2)


def rotate(x, pos, inv_freq, interleaved):
    """x [T, H, D] bf16, pos [T] -> bf16, in 64 bits and rounded once."""
    if inv_freq is None or inv_freq.numel() == 0:
        return x.clone()
    half = inv_freq.numel()
    ang = pos.double()[:, None] * inv_freq.double()[None]
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    y = x.double()
    out = y.clone()
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        out[..., :half], out[..., half:2 * half] = a * c - b * s, b * c + a * s
    return out.float().to(torch.bfloat16)


# ---- attention -----------------------------------------------------------------

def attend(q, k, v, seen, scale):
    """q [n, Hq, D], k, v [L, Hkv, D] fp64, seen [n, L] -> (out, bound) fp64."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    if L == 0 or n == 0:
        return out, bound
    rows = seen.any(1)
    for h in range(Hq):
        kh, vh = k[:, h * Hkv // Hq], v[:, h * Hkv // Hq]
        s = torch.where(seen, (q[:, h] @ kh.T) * scale, -np.inf)
        mag = torch.where(seen, (q[:, h].abs() @ kh.abs().T) * scale, 0.0)
        p = torch.where(rows[:, None], torch.softmax(torch.where(rows[:, None], s, 0.0), -1), 0.0)
        vz = torch.where(seen.any(0)[:, None], vh, 0.0)
        out[:, h] = p @ vz
        delta = (D * F * mag).amax(1) + 2 * F * (torch.where(seen, s.abs(), 0.0).amax(1) + 1)
        e = (p @ vz.abs()) * (U + 2 * delta + L * F)[:, None]
        bound[:, h] = U * (out[:, h].abs() + e) + e
    return out, bound


def prompt(q, k, v, lens, scale, gy=None):
    """Packed causal attention in fp64 on the host.  Returns {name: (value,
    bound)} of out and, with gy, grad_q, grad_k, grad_v."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    q, k, v = q.double(), k.double(), v.double()
    names = ("out", "grad_q", "grad_k", "grad_v")
    val = {n: torch.zeros_like(q if n in ("out", "grad_q") else k) for n in names}
    err = {n: torch.zeros_like(val[n]) for n in names}
    at = 0
    for n in lens:
        r = slice(at, at + n)
        at += n
        if n == 0:
            continue
        seen = torch.arange(n)[None] <= torch.arange(n)[:, None]
        val["out"][r], err["out"][r] = attend(q[r], k[r], v[r], seen, scale)
        if gy is None:
            continue
        g = gy[r].double()
        for h in range(Hq):
            hk = h // G
            qh, kh, vh, gh = q[r][:, h], k[r][:, hk], v[r][:, hk], g[:, h]
            s = torch.where(seen, (qh @ kh.T) * scale, -np.inf)
            mag = torch.where(seen, (qh.abs() @ kh.abs().T) * scale, 0.0)
            p = torch.softmax(s, -1)
            top = torch.where(seen, s.abs(), 0.0)
            # of a weight recomputed from the score and the row's log-sum-exp
            ep = D * F * mag + 2 * F * (top + 1) + ((D * F * mag).amax(1) + 4 * F * (top.amax(1) + 1) + n * F)[:, None]
            val["grad_v"][r][:, hk] += p.T @ gh
            err["grad_v"][r][:, hk] += (p * (U + ep + n * F)).T @ gh.abs()
            dp = gh @ vh.T
            delta = (p * dp).sum(-1, keepdim=True)
            e_delta = (gh.abs() * (err["out"][r][:, h] + D * F * val["out"][r][:, h].abs())).sum(-1, keepdim=True)
            e_dp = D * F * (gh.abs() @ vh.abs().T)
            ds = torch.where(seen, p * (dp - delta), 0.0)
            # the sums below run over fp32 products of rounded score gradients
            e_ds = torch.where(seen, ds.abs() * (U + ep + n * F) + (1 + U) * p * (1 + ep) * (e_dp + e_delta), 0.0)
            val["grad_q"][r][:, h] = scale * (ds @ kh)
            err["grad_q"][r][:, h] = scale * (e_ds @ kh.abs())
            val["grad_k"][r][:, hk] += scale * (ds.T @ qh)
            err["grad_k"][r][:, hk] += scale * (e_ds.T @ qh.abs())
    for name in names[1:]:
        err[name] = U * (val[name].abs() + err[name]) + err[name]
    return {n: (val[n], err[n]) for n in (names if gy is not None else names[:1])}


def within(got, want, bound, what):
    g = got.detach().cpu().double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    assert torch.isfinite(g).all(), f"{what}: non-finite values"
    over = (g - want).abs() - bound
    assert float(over.max() if over.numel() else 0.0) <= 1e-30, (
        f"{what}: over the rounding bound by {float(over.max()):.3e} at {np.unravel_index(int(over.argmax()), over.shape)}")


def offsets_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def normal(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


# ---- a cache on the host -----------------------------------------------------------

class HostCache:
    """Page table, codes and scales of sequences of the given lengths, filled
    with garbage (NaN scales) where no token lies."""

    def __init__(self, lens, kv_heads, page, D, seed=0, spare=2, width=None):
        g = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.page, self.D, self.H = page, D, kv_heads
        self.pages = sum(need) + spare
        self.width = max([1, *need]) if width is None else width
        order = g.permutation(self.pages)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, kv_heads, page)
        self.k_codes, self.v_codes = (torch.from_numpy(g.integers(0, 256, (*shape, D // 2), dtype=np.uint8)) for _ in "kv")
        self.k_scale, self.v_scale = (torch.full((*shape, D // 64), float("nan")) for _ in "kv")

    def put(self, b, pos, k, v):
        """k, v [H, D] bf16 of token pos of sequence b."""
        pg, i = int(self.table[b, pos // self.page]), pos % self.page
        self.k_codes[pg, :, i], self.k_scale[pg, :, i] = encode(k)
        self.v_codes[pg, :, i], self.v_scale[pg, :, i] = encode(v)

    def fill(self, lens, seed):
        for b, n in enumerate(lens):
            k, v = normal(seed + 2 * b, n, self.H, self.D), normal(seed + 2 * b + 1, n, self.H, self.D)
            for p in range(n):
                self.put(b, p, k[p], v[p])

    def dense(self, b, n):
        """(k, v) fp64 [n, H, D] of the first n tokens of sequence b."""
        pg = torch.from_numpy(self.table[b].astype(np.int64))
        out = []
        for codes, scale in ((self.k_codes, self.k_scale), (self.v_codes, self.v_scale)):
            x = decode(codes[pg.clamp(min=0)], scale[pg.clamp(min=0)])       # [w, H, page, D]
            out.append(x.transpose(1, 2).flatten(0, 1)[:n])
        return out

    def to(self, dev):
        from nf4_bit_weight_amd import NF4KVCache
        return (NF4KVCache(*(t.to(dev) for t in (self.k_codes, self.k_scale, self.v_codes, self.v_scale))),
                torch.from_numpy(self.table).to(dev))
