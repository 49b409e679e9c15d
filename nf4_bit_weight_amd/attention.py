"""Attention between the quantised projections: a paged key/value cache held in
4 bits, attention over it, and causal attention over packed prompts (the C ABI
of include/nf4_attn.h).

As in `api`, argument marshalling only, here in the compiled module _nf4_torch
(csrc/nf4_torch.cpp): tensors are checked, their pointers and the current
stream of their device are passed on, and a non-zero status raises NF4Error.

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

No call has a forward derivative: inputs with a forward-mode tangent are refused.
The cache calls have no gradient: while gradients are recorded, inputs that
require one are refused (detach them, or call under torch.no_grad()); a training
step rotates in torch.  nf4_prompt_attention_fwd and _bwd are the two halves that
autograd.nf4_prompt_attention records; called by themselves they record nothing,
like nf4_matmul_fwd.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib as L

_SIZE_MAX = 2 ** 64 - 1
_ext = None


def _call(name: str, *args):
    """One call of the compiled module; its int is the status of a refusal."""
    global _ext
    if _ext is None:
        L.lib()
        from . import _nf4_torch as _ext      # raises if it has not been built
    r = getattr(_ext, name)(*args)
    if type(r) is int:
        L.check("nf4_" + _C_NAMES.get(name, name), r)
    return r


_C_NAMES = {"prompt_fwd": "prompt_attention_fwd", "prompt_bwd": "prompt_attention_bwd",
            "prompt_attention": "prompt_attention_fwd", "route": "route_fwd", "expert_combine": "expert_combine_fwd",
            "int8_grouped": "int8_grouped_matmul"}


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
    codes = [torch.zeros((*shape, head_dim // 2), dtype=torch.uint8, device=device) for _ in range(2)]
    scale = [torch.zeros((*shape, head_dim // 64), dtype=torch.float32, device=device) for _ in range(2)]
    return NF4KVCache(codes[0], scale[0], codes[1], scale[1])


def nf4_kv_append(cache: NF4KVCache, k: torch.Tensor, v: torch.Tensor, lengths: torch.Tensor,
                  page_table: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                  inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False,
                  q: Optional[torch.Tensor] = None, return_k: bool = False,
                  q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Put new keys and values into the cache, keys turned by their positions
    (inv_freq float32 [rotary / 2]; pairs (i, i + rotary / 2), or neighbours with
    `interleaved`).  Returns (q turned alike or None, the turned bf16 keys with
    `return_k` or None)."""
    return _call("kv_append", cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale, k, v, lengths, page_table,
                 offsets, inv_freq, interleaved, q, return_k, q_out, k_out)


def nf4_kv_dequantize(cache: NF4KVCache, lengths: torch.Tensor, page_table: torch.Tensor,
                      offsets: Optional[torch.Tensor] = None, rows: Optional[int] = None,
                      k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None):
    """The keys and values that the cache stands for, bf16 [rows, Hkv, D]: of the
    last offsets[b+1] - offsets[b] tokens of each sequence (without offsets, the
    last one).  `rows` is the number of rows of the result."""
    return _call("kv_dequantize", cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale, lengths, page_table,
                 offsets, rows, k_out, v_out)


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
    return _call("kv_attention", cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale, q, lengths, page_table,
                 offsets, scale, out, ws)


def nf4_prompt_attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor,
                             scale: Optional[float] = None, out: Optional[torch.Tensor] = None, for_backward: bool = False):
    """Causal attention inside each packed sequence.  Returns out, or with
    for_backward what the backward call takes: (out, out_rest, lse), out_rest
    bf16 like out and lse float32 [Hq, T]."""
    return _call("prompt_fwd", q, k, v, offsets, scale, out, for_backward)


def nf4_prompt_attention_bwd(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             out: torch.Tensor, out_rest: Optional[torch.Tensor], lse: torch.Tensor,
                             offsets: torch.Tensor, scale: Optional[float] = None, ws: Optional[torch.Tensor] = None):
    """(grad_q, grad_k, grad_v) from the forward call's inputs and results."""
    return _call("prompt_bwd", grad_out, q, k, v, out, out_rest, lse, offsets, scale, ws)
