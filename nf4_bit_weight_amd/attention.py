"""Attention between the quantised projections: a paged key/value cache held in
4 bits, attention over it, and causal attention over packed prompts (the C ABI
of include/nf4_attn.h).

As in `api`, argument marshalling only: tensors are checked, their pointers and
the current stream of their device are passed on, and a non-zero status raises
NF4Error.

Tensor conventions (all on one CUDA/HIP device):
  q               bfloat16 [T, Hq, D]; k, v  bfloat16 [T, Hkv, D]; D is 64 or 128
                  and Hq a multiple of Hkv.  The heads of a row are contiguous;
                  the rows may be strided (a slice of a joint projection), by a
                  multiple of 8 elements
  offsets         int32 [B + 1], rows offsets[b] .. offsets[b+1]-1 belong to
                  sequence b; for the cache calls None means one row each
  lengths         int32 [B], tokens of each sequence with the rows of the call
  page_table      int32 [B, width], the pages that hold a sequence's tokens
Rows outside every sequence are zeros in a result allocated here and left as
they were in one that is passed in.
"""

from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib as L
from .api import _need, _ptr

_BLOCK = 64
_SIZE_MAX = 2 ** 64 - 1
_BF16, _U8, _F32, _I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
_current_device = torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


@dataclass
class NF4KVCache:
    """A paged key/value cache held in 4 bits (layout and encoding in
    nf4_attn.h): every vector of D elements is D/2 bytes of fp4 (e2m1) patterns
    and one fp32 scale per 64 elements."""
    k_codes: torch.Tensor      # uint8   [P, Hkv, page, D / 2]
    k_scale: torch.Tensor      # float32 [P, Hkv, page, D / 64]
    v_codes: torch.Tensor
    v_scale: torch.Tensor

    @property
    def pages(self) -> int:
        return self.k_codes.shape[0]

    @property
    def kv_heads(self) -> int:
        return self.k_codes.shape[1]

    @property
    def page_size(self) -> int:
        return self.k_codes.shape[2]

    @property
    def head_dim(self) -> int:
        return 2 * self.k_codes.shape[3]

    def tensors(self):
        return self.k_codes, self.k_scale, self.v_codes, self.v_scale

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.tensors())


def nf4_kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> NF4KVCache:
    """An empty cache (zeros) of `pages` pages of `page_size` tokens."""
    if head_dim not in (64, 128):
        raise ValueError(f"head_dim must be 64 or 128, got {head_dim}")
    if page_size < 16 or page_size % 16:
        raise ValueError(f"page_size must be a multiple of 16, got {page_size}")
    if pages < 0 or kv_heads < 1:
        raise ValueError("pages must be at least 0 and kv_heads at least 1")
    shape = (pages, kv_heads, page_size)
    codes = [torch.zeros((*shape, head_dim // 2), dtype=_U8, device=device) for _ in range(2)]
    scale = [torch.zeros((*shape, head_dim // _BLOCK), dtype=_F32, device=device) for _ in range(2)]
    return NF4KVCache(codes[0], scale[0], codes[1], scale[1])


def _cache_args(c: NF4KVCache):
    kc, ks, vc, vs = c.k_codes, c.k_scale, c.v_codes, c.v_scale
    shape, dev = kc.shape, kc.device
    if len(shape) != 4:
        raise ValueError("k_codes must be [pages, kv_heads, page, head_dim / 2]")
    P, H, page, half = shape
    if half != 64 and half != 32:
        raise ValueError(f"the cache's head_dim must be 64 or 128, got {2 * half}")
    if page < 16 or page % 16:
        raise ValueError(f"the cache's page must be a multiple of 16 tokens, got {page}")
    n = P * H * page * half
    _need(kc, "k_codes", _U8)
    _need(vc, "v_codes", _U8, n, dev)
    _need(ks, "k_scale", _F32, n // 32, dev)
    _need(vs, "v_scale", _F32, n // 32, dev)
    return dev, H, 2 * half, (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), P, page, H, 2 * half)


def _seq_args(rows: int, lengths, page_table, offsets, device):
    _need(lengths, "lengths", _I32, device=device)
    _need(page_table, "page_table", _I32, device=device)
    table, B = page_table.shape, lengths.numel()
    if len(table) != 2 or lengths.dim() != 1 or table[0] != B:
        raise ValueError("lengths must be [B] and page_table [B, width]")
    if offsets is None:
        if rows != B:
            raise ValueError(f"without offsets there is one row per sequence: {rows} rows, {B} sequences")
        return None, lengths.data_ptr(), B, page_table.data_ptr(), table[1]
    _need(offsets, "offsets", _I32, B + 1, device)
    return offsets.data_ptr(), lengths.data_ptr(), B, page_table.data_ptr(), table[1]


def _rows(t: torch.Tensor, name: str, heads: Optional[int], D: int, device, rows: Optional[int] = None) -> int:
    """Check a [T, heads, D] bf16 tensor with free row stride; its stride."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != D or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [T, {'heads' if heads is None else heads}, {D}], got {tuple(shape)}")
    T, H = shape[0], shape[1]
    if rows is not None and T != rows:
        raise ValueError(f"{name} has {T} rows, expected {rows}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if T * H == 0:
        return 0
    sr, sh, sd = t.stride()
    if sd != 1 or (sh != D and H > 1) or (sr % 8 and T > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous and rows a multiple of 8 elements apart")
    return sr if T > 1 else 0


def _result(t: Optional[torch.Tensor], name: str, T: int, H: int, D: int, device):
    """(result tensor, whether rows outside every sequence are to be filled)."""
    if t is None:
        return torch.empty(T, H, D, dtype=_BF16, device=device), 1
    _need(t, name, _BF16, T * H * D, device)
    return t, 0


class _on:
    """The device of the tensors made current for a launch, if it is not, and
    the handle of its current stream."""

    __slots__ = ("index", "guard")

    def __init__(self, device):
        self.index = device.index
        self.guard = None if _current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return _current_stream(self.index)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _scale(scale: Optional[float], D: int) -> float:
    s = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if not (s > 0 and math.isfinite(s)):
        raise ValueError(f"scale must be positive and finite, got {scale}")
    return s


def nf4_kv_append(cache: NF4KVCache, k: torch.Tensor, v: torch.Tensor, lengths: torch.Tensor,
                  page_table: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                  inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False,
                  q: Optional[torch.Tensor] = None, return_k: bool = False,
                  q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Put new keys and values into the cache, keys turned by their positions
    (inv_freq float32 [rotary / 2]; pairs (i, i + rotary / 2), or neighbours with
    `interleaved`).  Returns (q turned alike or None, the turned bf16 keys with
    `return_k` or None)."""
    dev, H, D, cargs = _cache_args(cache)
    ks = _rows(k, "k", H, D, dev)
    T = k.shape[0]
    vs = _rows(v, "v", H, D, dev, T)
    sargs = _seq_args(T, lengths, page_table, offsets, dev)
    rotary = 0
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", _F32, device=dev)
        rotary = 2 * inv_freq.numel()
        if rotary > D or rotary % 16:
            raise ValueError(f"inv_freq must have a multiple of 8 elements, at most {D // 2}, got {inv_freq.numel()}")
    Hq, qs, fill = H, 0, 1
    if q is not None:
        qs = _rows(q, "q", None, D, dev, T)
        Hq = q.shape[1]
        if Hq < 1 or Hq % H:
            raise ValueError(f"{Hq} query heads do not divide over {H} key heads")
        q_out, fill = _result(q_out, "q_out", T, Hq, D, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k_out is not None or return_k:
        k_out, kfill = _result(k_out, "k_out", T, H, D, dev)
        if q is not None and kfill != fill:
            raise ValueError("pass both of q_out and k_out, or neither")
        fill = kfill
    with _on(dev) as stream:
        st = L.lib().nf4_kv_append(_ptr(q), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, Hq, *sargs, _ptr(inv_freq), rotary,
                                   int(interleaved), *cargs, _ptr(q_out), _ptr(k_out), fill, stream)
    L.check("nf4_kv_append", st)
    return q_out, k_out


def nf4_kv_dequantize(cache: NF4KVCache, lengths: torch.Tensor, page_table: torch.Tensor,
                      offsets: Optional[torch.Tensor] = None, rows: Optional[int] = None,
                      k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None):
    """The keys and values that the cache stands for, bf16 [rows, Hkv, D]: of the
    last offsets[b+1] - offsets[b] tokens of each sequence (without offsets, the
    last one).  `rows` is the number of rows of the result."""
    dev, H, D, cargs = _cache_args(cache)
    if rows is None:
        if offsets is not None:
            raise ValueError("with offsets, pass the number of rows")
        rows = lengths.shape[0]
    if rows < 0:
        raise ValueError(f"rows must not be negative, got {rows}")
    sargs = _seq_args(rows, lengths, page_table, offsets, dev)
    if (k_out is None) != (v_out is None):
        raise ValueError("pass both of k_out and v_out, or neither")
    k_out, fill = _result(k_out, "k_out", rows, H, D, dev)
    v_out, _ = _result(v_out, "v_out", rows, H, D, dev)
    with _on(dev) as stream:
        st = L.lib().nf4_kv_dequantize(rows, *sargs, *cargs, k_out.data_ptr(), v_out.data_ptr(), fill, stream)
    L.check("nf4_kv_dequantize", st)
    return k_out, v_out


def nf4_kv_attention_workspace(T: int, B: int, Hq: int, Hkv: int, D: int, width: int, page: int) -> int:
    """Bytes that nf4_kv_attention wants for T rows in B sequences whose page
    tables are `width` pages of `page` tokens wide."""
    n = L.lib().nf4_kv_attention_workspace(T, B, Hq, Hkv, D, width, page)
    if n == _SIZE_MAX:
        raise ValueError(f"unsupported sizes: T {T}, B {B}, heads {Hq} on {Hkv}, D {D}, table {width} x {page}")
    return n


def nf4_kv_attention(q: torch.Tensor, cache: NF4KVCache, lengths: torch.Tensor, page_table: torch.Tensor,
                     offsets: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of the newest rows of each sequence over its cached tokens, each
    row seeing the tokens up to its own (scale 1/sqrt(D) unless given)."""
    dev, H, D, cargs = _cache_args(cache)
    qs = _rows(q, "q", None, D, dev)
    T, Hq = q.shape[0], q.shape[1]
    if Hq < 1 or Hq % H:
        raise ValueError(f"{Hq} query heads do not divide over {H} key heads")
    sargs = _seq_args(T, lengths, page_table, offsets, dev)
    s = _scale(scale, D)
    out, fill = _result(out, "out", T, Hq, D, dev)
    with _on(dev) as stream:
        if ws is None:
            need = nf4_kv_attention_workspace(T, sargs[2], Hq, H, D, sargs[4], cargs[5])
            ws = torch.empty(need, dtype=_U8, device=dev) if need else None
        else:
            _need(ws, "ws", device=dev)
        st = L.lib().nf4_kv_attention(q.data_ptr(), qs, T, Hq, *sargs, *cargs, s, out.data_ptr(), fill, _ptr(ws),
                                      0 if ws is None else ws.numel() * ws.element_size(), stream)
    L.check("nf4_kv_attention", st)
    return out


def _prompt_args(q, k, v, offsets):
    D = q.shape[2] if q.dim() == 3 else 0
    if D not in (64, 128):
        raise ValueError(f"q must be [T, Hq, D] with D 64 or 128, got {tuple(q.shape)}")
    dev = q.device
    qs = _rows(q, "q", None, D, dev)
    T, Hq = q.shape[0], q.shape[1]
    ks = _rows(k, "k", None, D, dev, T)
    H = k.shape[1]
    vs = _rows(v, "v", H, D, dev, T)
    if H < 1 or Hq < 1 or Hq % H:
        raise ValueError(f"{Hq} query heads do not divide over {H} key heads")
    _need(offsets, "offsets", _I32, device=dev)
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets must be [B + 1]")
    return dev, T, offsets.numel() - 1, Hq, H, D, (q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs)


def nf4_prompt_attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor,
                             scale: Optional[float] = None, out: Optional[torch.Tensor] = None, for_backward: bool = False):
    """Causal attention inside each packed sequence.  Returns out, or with
    for_backward what the backward call takes: (out, out_rest, lse), out_rest
    bf16 like out and lse float32 [Hq, T]."""
    dev, T, B, Hq, H, D, ptrs = _prompt_args(q, k, v, offsets)
    s = _scale(scale, D)
    out, fill = _result(out, "out", T, Hq, D, dev)
    rest = lse = None
    if for_backward:
        rest = torch.empty((T, Hq, D), dtype=_BF16, device=dev)
        lse = torch.empty((Hq, T), dtype=_F32, device=dev)
    with _on(dev) as stream:
        st = L.lib().nf4_prompt_attention_fwd(*ptrs, T, offsets.data_ptr(), B, Hq, H, D, s, out.data_ptr(), _ptr(rest),
                                              _ptr(lse), fill, stream)
    L.check("nf4_prompt_attention_fwd", st)
    return (out, rest, lse) if for_backward else out


def nf4_prompt_attention_bwd(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             out: torch.Tensor, out_rest: Optional[torch.Tensor], lse: torch.Tensor,
                             offsets: torch.Tensor, scale: Optional[float] = None, ws: Optional[torch.Tensor] = None):
    """(grad_q, grad_k, grad_v) from the forward call's inputs and results."""
    dev, T, B, Hq, H, D, ptrs = _prompt_args(q, k, v, offsets)
    s = _scale(scale, D)
    gs = _rows(grad_out, "grad_out", Hq, D, dev, T)
    _need(out, "out", _BF16, T * Hq * D, dev)
    _need(out_rest, "out_rest", _BF16, T * Hq * D, dev)
    _need(lse, "lse", _F32, T * Hq, dev)
    gq = torch.empty((T, Hq, D), dtype=_BF16, device=dev)
    gk = torch.empty((T, H, D), dtype=_BF16, device=dev)
    gv = torch.empty((T, H, D), dtype=_BF16, device=dev)
    with _on(dev) as stream:
        if ws is None:
            need = int(L.lib().nf4_prompt_attention_bwd_workspace(T, B, Hq, H, D))
            ws = torch.empty(need, dtype=_U8, device=dev)
        else:
            _need(ws, "ws", device=dev)
        st = L.lib().nf4_prompt_attention_bwd(grad_out.data_ptr(), gs, *ptrs, out.data_ptr(), _ptr(out_rest),
                                              lse.data_ptr(), T, offsets.data_ptr(), B, Hq, H, D, s, gq.data_ptr(),
                                              gk.data_ptr(), gv.data_ptr(), 1, ws.data_ptr(),
                                              ws.numel() * ws.element_size(), stream)
    L.check("nf4_prompt_attention_bwd", st)
    return gq, gk, gv
