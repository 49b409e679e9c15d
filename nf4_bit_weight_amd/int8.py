"""Linear layers in 8-bit integers with a scale for each output channel and each
token (the C ABI of include/nf4_int8.h): the form for serving, beside the
blockwise 8-bit formats of `api`, which multiply in bf16 and train.

As in `attention`, argument marshalling only, in the compiled module _nf4_torch
(csrc/nf4_torch_experts.cpp).  Activations are float32 or bfloat16 [M, K], the
elements of a row contiguous, the rows strided as they like; or an NF4Int8, for
activations that several layers share.  The calls have no gradient (rounding has none): while
gradients are recorded, inputs that require one are refused (detach them, or call
under torch.no_grad()).
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Union

import torch

from . import _lib as L
from .attention import _call

_SIZE_MAX = 2 ** 64 - 1


@dataclass
class NF4Int8:
    """N rows of K integers with a scale each: a weight [N, K] (one row for each
    output channel), or N quantised tokens.  `q` has K rounded up to a multiple of
    128 columns, zeros behind K."""
    q: torch.Tensor            # int8    [N, row bytes]
    scale: torch.Tensor        # float32 [N]
    N: int
    K: int

    def per_expert(self, E: int) -> "NF4Int8":
        """View of an [E*N, K] stack with N rows per expert (the form the grouped
        call takes)."""
        if self.N % E:
            raise ValueError(f"{self.N} rows do not split into {E} experts")
        return NF4Int8(self.q, self.scale, self.N // E, self.K)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.q, self.scale))


def nf4_int8_quantize(x: torch.Tensor) -> NF4Int8:
    """x [N, K] (float32 or bfloat16), weight or activations, to integers by rows."""
    q, scale = _call("int8_quantize", x)
    return NF4Int8(q, scale, x.shape[0], x.shape[1])


def _x(x, w: NF4Int8):
    if isinstance(x, NF4Int8):
        if x.K != w.K:
            raise ValueError(f"x has rows of {x.K}, the weight of {w.K}")
        return x.q, x.scale
    return x, None


def nf4_int8_workspace(x: Union[torch.Tensor, NF4Int8], w: NF4Int8, rows: Optional[int] = None, E: int = 0) -> int:
    """Bytes of workspace that the product of x and w wants (`rows` of y and E
    experts for the grouped one)."""
    ready = isinstance(x, NF4Int8)
    M = x.q.shape[0] if ready else x.shape[0]
    kind = L.NF4_DTYPE_I8 if ready else L.NF4_DTYPE_BF16 if x.dtype == torch.bfloat16 else L.NF4_DTYPE_F32
    n = L.lib().nf4_int8_workspace(kind, M, M if rows is None else rows, w.N, w.K, E)
    if n == _SIZE_MAX:
        raise ValueError(f"unsupported sizes: M {M}, N {w.N}, K {w.K}, E {E}")
    return n


def nf4_int8_matmul(x: Union[torch.Tensor, NF4Int8], w: NF4Int8, bias: Optional[torch.Tensor] = None,
                    out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] = x . W^T + bias (float32 [N]), the tokens of x quantised on the
    way.  out_dtype is float32 or bfloat16: x's own, or bfloat16 for an NF4Int8."""
    xq, xs = _x(x, w)
    return _call("int8_matmul", xq, xs, w.q, w.scale, w.N, w.K, bias, out_dtype, out, ws)


def nf4_int8_grouped_matmul(x: Union[torch.Tensor, NF4Int8], offsets: torch.Tensor, w: NF4Int8, E: int,
                            tokens: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                            out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Per-expert y over expert-sorted rows; w is the [E*N, K] stack (N per expert).
    With `tokens` (a routing's) row r of y takes row tokens[r] of x, so that no
    gathered copy of x is made.  Rows behind offsets[E] are zeros in a result
    allocated here and left as they were in one that is passed in."""
    xq, xs = _x(x, w)
    return _call("int8_grouped", xq, xs, w.q, w.scale, w.N, w.K, None, out_dtype, out, ws, offsets, E, tokens)
