"""Products in 8-bit integers against exact sums: the integers are compared
whole, outputs to the roundings of their last steps."""

import math

import numpy as np
import pytest
import torch

import expert_ref as R
from nf4_bit_weight_amd import NF4Int8, nf4_int8_grouped_matmul, nf4_int8_matmul, nf4_int8_quantize, nf4_int8_workspace
from nf4_bit_weight_amd._lib import NF4Error

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def check_rows(got: NF4Int8, x):
    q, s = R.quantize(x)
    K = x.shape[1]
    assert got.q.shape == (x.shape[0], -(-K // 128) * 128) and (got.N, got.K) == tuple(x.shape)
    assert torch.equal(got.q[:, :K].cpu().long(), q)
    assert not got.q[:, K:].any()
    assert torch.equal(torch.nan_to_num(got.scale.cpu(), nan=-1.0), torch.nan_to_num(s, nan=-1.0))


@pytest.mark.parametrize("M,K", [(1, 1), (3, 16), (5, 127), (2, 128), (4, 129), (7, 1000), (2, 4096), (3, 5120), (2, 14336), (1, 40001), (1, 130944)])
@pytest.mark.parametrize("dtype", R.BOTH)
def test_quantize(M, K, dtype):
    x = (R.normal(M + K, M, K) * torch.exp(R.normal(K, K))).to(dtype)
    check_rows(nf4_int8_quantize(x.to(DEV)), x)
    if K > 8:
        wide = torch.cat((x, x), 1).to(DEV)
        check_rows(nf4_int8_quantize(wide[:, 3:K]), wide[:, 3:K].cpu())            # strided, not aligned
        check_rows(nf4_int8_quantize(wide[:, :K]), x)


@pytest.mark.parametrize("dtype", R.BOTH)
def test_quantize_edges(dtype):
    """Half-way values go to the even integer; values a step beside them do not."""
    K = 512
    half = torch.arange(K, dtype=torch.float64) % 127 + 0.5
    rows = []
    for top in (127.0, 254.0, 31.75, 2.0 ** -100, 127.0 * 2.0 ** 100):
        x = (half * top / 127).to(dtype)
        for step in (0, 1, -1):
            y = x if step == 0 else torch.nextafter(x, torch.tensor(math.inf * step, dtype=dtype))
            y = torch.where(torch.arange(K) % 2 == 0, y, -y)
            y[7] = top
            rows.append(y)
    for top in (1.0, 3.0, 0.7, 1e30):                          # tops whose 127th is no short number
        x = (half * top / 127).to(dtype)
        x[7] = -top
        rows.append(x)
    lowest, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    for v in (0.0, tiny, 2.0 ** -119, 2.0 ** -120, 1e-40, lowest):
        y = torch.zeros(K, dtype=dtype)
        y[5], y[9] = v, -v / 2
        rows.append(y)
    for v in (math.nan, math.inf, -math.inf):
        y = torch.ones(K, dtype=dtype)
        y[300] = v
        rows.append(y)
    x = torch.stack(rows)
    check_rows(nf4_int8_quantize(x.to(DEV)), x)


SHAPES = [(1, 1, 1), (1, 16, 64), (1, 4096, 4096), (2, 100, 300), (3, 33, 128), (8, 1000, 640), (16, 129, 4096), (17, 64, 200), (31, 500, 1024),
          (32, 1024, 2048), (33, 77, 129), (64, 256, 512), (65, 300, 384), (100, 1024, 1152), (128, 128, 4096), (129, 257, 640),
          (200, 4096, 256), (256, 256, 128), (300, 513, 5120), (512, 1024, 1024), (700, 1000, 777), (1024, 2048, 512), (2048, 640, 896),
          # every shape of tile, whole and with parts; K of one step, of fewer than are in flight, of more
          (512, 4096, 128), (1000, 4100, 500), (1024, 4096, 640), (520, 4000, 1000), (2048, 4096, 128), (2048, 4000, 300),
          (4096, 4096, 256), (2500, 3500, 700),
          # few rows: channels 16, 32 and 64 a workgroup, K in one to eight parts and beyond what is in flight
          (5, 14336, 1100), (3, 14336, 128), (16, 7300, 384), (1, 15000, 600), (20, 4096, 1300), (33, 8100, 2200), (50, 1000, 8000), (64, 4096, 200), (2, 40, 20000)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(M, N, K):
    x, w, b = R.normal(M + K, M, K), 0.05 * R.normal(N, N, K), R.normal(3, N)
    qw, sw = R.quantize(w)
    weight = nf4_int8_quantize(w.to(DEV))
    for i, dtype in enumerate(R.BOTH):
        xd = x.to(dtype)
        q, s = R.quantize(xd)
        bias = b if i else None
        want, bound = R.product(q, s, qw, sw, bias)
        for out_dtype in R.BOTH:
            y = nf4_int8_matmul(xd.to(DEV), weight, bias=None if bias is None else bias.to(DEV), out_dtype=out_dtype)
            assert y.dtype == out_dtype
            R.within(y, want, R.rounded(bound, want, out_dtype), f"{M} {N} {K} {dtype} {out_dtype}")
        ready = nf4_int8_quantize(xd.to(DEV))
        assert torch.equal(nf4_int8_matmul(ready, weight, bias=None if bias is None else bias.to(DEV), out_dtype=out_dtype), y)


def random_bytes(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).integers(-128, 128, shape, dtype=np.int8))


@pytest.mark.parametrize("M,N,K", [(1, 40, 130944), (20, 40, 130944), (70, 130, 4096), (300, 300, 1024)])
def test_matmul_sums_are_exact(M, N, K):
    """Integers of either sign up to the ends of their range, sums up to 2^31 - 1."""
    x, w = random_bytes(1, M, K), random_bytes(2, N, K)
    x[0], w[0] = -128, -128
    w[1] = 127
    one = lambda n: torch.ones(n, device=DEV)
    y = nf4_int8_matmul(NF4Int8(x.to(DEV), one(M), M, K), NF4Int8(w.to(DEV), one(N), N, K), out_dtype=torch.float32)
    want = (x.double() @ w.double().T)
    assert torch.equal(y.cpu(), want.float())


def test_matmul_special_rows_and_channels():
    M, N, K = 40, 48, 256
    x, w = R.normal(1, M, K), R.normal(2, N, K)
    x[3], x[5, 7], x[6, 9] = 0.0, math.nan, math.inf
    w[4], w[8, 1] = 0.0, math.nan
    y = nf4_int8_matmul(x.to(DEV), nf4_int8_quantize(w.to(DEV))).cpu()
    bad = torch.zeros((M, N), dtype=torch.bool)
    bad[5] = bad[6] = True
    bad[:, 8] = True
    assert torch.equal(torch.isnan(y), bad)
    clean = y.masked_fill(bad, 1.0)
    assert bool((clean[3, :8] == 0).all()) and bool((clean[:5, 4] == 0).all())
    big = nf4_int8_matmul(torch.full((2, K), 3e38, device=DEV), nf4_int8_quantize(torch.full((N, K), 1e-3, device=DEV)))
    assert torch.isfinite(big).all() or float(3e38 * 1e-3 * K) > 3e38


def test_matmul_strides_outputs_and_empty_sizes():
    M, N, K = 37, 96, 200
    x, w = R.normal(1, M, 2 * K).to(DEV), nf4_int8_quantize(R.normal(2, N, K).to(DEV))
    want = nf4_int8_matmul(x[:, :K].contiguous(), w)
    assert torch.equal(nf4_int8_matmul(x[:, :K], w), want)
    out = torch.full((M, N), 9.0, device=DEV)
    ws = torch.empty(nf4_int8_workspace(x[:, :K], w), dtype=torch.uint8, device=DEV)
    assert nf4_int8_matmul(x[:, :K], w, out=out, ws=ws) is out and torch.equal(out, want)
    assert torch.equal(nf4_int8_matmul(x[:1, :K].expand(M, K), w), want[:1].expand(M, N))
    assert nf4_int8_matmul(torch.empty((0, K), device=DEV), w).shape == (0, N)
    empty = nf4_int8_quantize(torch.empty((N, 0), device=DEV))
    b = R.normal(3, N).to(DEV)
    assert torch.equal(nf4_int8_matmul(torch.empty((M, 0), device=DEV), empty, bias=b), b.expand(M, N))
    assert torch.equal(nf4_int8_matmul(torch.empty((300, 0), device=DEV), empty), torch.zeros(300, N, device=DEV))
    none = nf4_int8_quantize(torch.empty((0, K), device=DEV))
    assert nf4_int8_matmul(x[:, :K], none).shape == (M, 0)


def grouped_case(seed, T, E, k, N, K, empty, dtype=torch.float32):
    e = R.random_experts(seed, T, E, k, empty)
    offsets, tokens, _ = R.plan(e, E)
    x, w = R.normal(seed + 1, T, K).to(dtype), 0.1 * R.normal(seed + 2, E * N, K)
    q, s = R.quantize(x)
    qw, sw = R.quantize(w)
    want, bound = torch.zeros((T * k, N), dtype=torch.float64), torch.zeros((T * k, N), dtype=torch.float64)
    for i in range(E):
        a, b = int(offsets[i]), int(offsets[i + 1])
        rows = tokens[a:b].long()
        want[a:b], bound[a:b] = R.product(q[rows], s[rows], qw[i * N:(i + 1) * N], sw[i * N:(i + 1) * N])
    return x, w, offsets, tokens, want, bound


GROUPED = [(1, 4, 2, 16, 64, 0), (3, 64, 8, 128, 256, 0), (5, 8, 1, 33, 100, 2), (40, 4, 2, 96, 384, 0), (64, 64, 8, 64, 128, 5), (200, 3, 1, 130, 640, 0),
           (130, 5, 2, 256, 512, 129), (300, 8, 2, 512, 256, 1), (257, 16, 4, 1024, 128, 0), (90, 60, 4, 40, 200, 3), (20, 200, 3, 8, 64, 0), (7, 4, 2, 64, 64, 7),
           (1500, 4, 2, 1000, 256, 10), (3000, 4, 2, 2000, 100, 0), (2100, 5, 1, 4000, 128, 100), (900, 1, 1, 300, 384, 0)]


@pytest.mark.parametrize("T,E,k,N,K,empty", GROUPED)
@pytest.mark.parametrize("dtype", R.BOTH)
def test_grouped(T, E, k, N, K, empty, dtype):
    x, w, offsets, tokens, want, bound = grouped_case(T + N, T, E, k, N, K, empty, dtype)
    weight = nf4_int8_quantize(w.to(DEV)).per_expert(E)
    xd, od, td = x.to(DEV), offsets.to(DEV), tokens.to(DEV)
    y = nf4_int8_grouped_matmul(xd, od, weight, E, tokens=td)
    assert y.dtype == dtype
    R.within(y, want, R.rounded(bound, want, dtype))
    n = int(offsets[-1])
    assert bool((y[n:] == 0).all())
    # rows gathered first, quantised before, and into a tensor of the caller's
    rows = xd[td.clamp(min=0).long()]
    assert torch.equal(nf4_int8_grouped_matmul(rows, od, weight, E), y)
    ready = nf4_int8_quantize(xd)
    out = torch.full((T * k, N), 5.0, dtype=torch.float32, device=DEV)
    assert nf4_int8_grouped_matmul(ready, od, weight, E, tokens=td, out_dtype=torch.float32, out=out) is out
    R.within(out[:n], want[:n], R.rounded(bound[:n], want[:n], torch.float32))
    assert bool((out[n:] == 5).all())


def test_grouped_malformed_arrays_stay_in_range():
    x, w, offsets, tokens, want, bound = grouped_case(5, 50, 6, 2, 64, 128, 0)
    weight, xd = nf4_int8_quantize(w.to(DEV)).per_expert(6), x.to(DEV)
    for bad in ([0, 10, 5, 200, -7, 90, 100], [-5, -4, -3, -2, -1, 0, 1], [100] * 7, [2 ** 31 - 1] * 7):
        y = nf4_int8_grouped_matmul(xd, torch.tensor(bad, dtype=torch.int32, device=DEV), weight, 6, tokens=tokens.to(DEV),
                                    out=torch.zeros((100, 64), device=DEV))
        assert y.shape == (100, 64)
    t = tokens.clone()
    t[3], t[9], t[20] = -4, 50, 2 ** 31 - 1
    y = nf4_int8_grouped_matmul(xd, offsets.to(DEV), weight, 6, tokens=t.to(DEV))
    keep = torch.ones(100, dtype=torch.bool)
    keep[[3, 9, 20]] = False
    R.within(y.cpu()[keep], want[keep], R.rounded(bound[keep], want[keep], torch.float32))


def test_refusals_on_the_device():
    w = nf4_int8_quantize(R.normal(1, 32, 128).to(DEV))
    x = torch.zeros((4, 128), device=DEV)
    with pytest.raises(ValueError, match="requires a gradient"):
        nf4_int8_matmul(x.clone().requires_grad_(), w)
    with pytest.raises(ValueError, match="requires a gradient"):
        nf4_int8_quantize(x.clone().requires_grad_())
    with torch.no_grad():
        assert nf4_int8_matmul(x.clone().requires_grad_(), w).shape == (4, 32)
    for bad, what in ((x[:, :64], "x must be"), (x.half(), "float32 or bfloat16"), (x.cpu(), "device"), (x[0], "two dimensions"),
                      (torch.zeros((128, 4), device=DEV).t(), "contiguous")):
        with pytest.raises(ValueError, match=what):
            nf4_int8_matmul(bad, w)
    for kw, what in ((dict(bias=torch.zeros(31, device=DEV)), "bias"), (dict(out_dtype=torch.float16), "out_dtype"), (dict(out_dtype=1), "out_dtype"),
                     (dict(out=torch.zeros((4, 31), device=DEV)), "out must be"), (dict(out=torch.zeros((4, 32), device=DEV).bfloat16()), "out must be"),
                     (dict(ws=torch.empty(8, dtype=torch.uint8)), "ws")):
        with pytest.raises(ValueError, match=what):
            nf4_int8_matmul(x, w, **kw)
    with pytest.raises(NF4Error, match="workspace|WORKSPACE"):
        nf4_int8_matmul(x, w, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(NF4Error):
        nf4_int8_quantize(torch.zeros((1, 130945), device=DEV))
    with pytest.raises(ValueError, match="rows of"):
        nf4_int8_matmul(nf4_int8_quantize(torch.zeros((2, 100), device=DEV)), w)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for kw, what in ((dict(E=0), "E must"), (dict(E=2), "weight"), (dict(E=1, offsets=off[:1]), "offsets"), (dict(E=1, tokens=off.long()), "tokens")):
        with pytest.raises(ValueError, match=what):
            nf4_int8_grouped_matmul(x, kw.pop("offsets", off), w, kw.pop("E"), **kw)
