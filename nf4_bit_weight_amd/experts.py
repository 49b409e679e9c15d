"""What stands around the grouped projections: a router's choice of experts, the
order in which the grouped calls take the rows, the tokens' rows to their
experts' places and back (the C ABI of include/nf4_experts.h).

As in `attention`, argument marshalling only, in the compiled module _nf4_torch
(csrc/nf4_torch_experts.cpp): tensors are checked, their pointers and the current
stream of their device are passed on, and a non-zero status raises NF4Error.

nf4_route is differentiable in the logits, nf4_expert_gather in x, and
nf4_expert_combine in the rows and the weights, once each.  They take any
floating dtype: float32 and bfloat16 as they are, others as float32; results and
gradients come back in the dtype that was passed in (weights are float32).  Sums
are float32.  No call has a forward derivative: inputs with a forward-mode tangent
are refused.  The *_bwd calls are the halves that autograd records; called by
themselves they record nothing.

Forward and backward can be captured into a graph together.  No eager graph of the
same leaves may live then: its gradient accumulators belong to the eager stream,
and autograd would draw that stream into the capture.  Leaves that are inputs of
these calls themselves are checked; for leaves further up, drop the eager results
before the capture.

    r = nf4_route(logits, 8)                                    # logits [T, E]
    rows = nf4_expert_gather(x, r)                              # [T * 8, H], sorted by expert
    h = nf4_grouped_linear(rows, r.offsets, w_up, E)            # or nf4_int8_grouped_matmul
    y = nf4_expert_combine(nf4_grouped_linear(act(h), r.offsets, w_down, E), r)

None of the calls here reads a row behind offsets[E].  The grouped calls of `api` and
`autograd` write none; nf4_int8_grouped_matmul writes zeros there in a result that it
allocates, and without `tokens` it quantises such rows of x with the others, which no
result sees.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from .attention import _call

_SCORES = {"softmax": False, "sigmoid": True}
_GROUP_SCORES = {"max": False, "top2": True}


@dataclass
class NF4Routing:
    """A choice of k experts for each of T tokens, and its plan (nf4_experts.h).
    Rows are the T * k rows that the experts take, sorted by expert and inside
    one by token; those behind offsets[E] belong to nobody.  The four integer results
    of nf4_route share one allocation of (3 T k + E + 1) numbers, which lives (and is saved
    by torch.save) as long as any of them: keep a clone() of one that is to outlive the rest."""
    weights: torch.Tensor      # float32 [T, k]
    experts: torch.Tensor      # int32   [T, k], -1: none
    offsets: torch.Tensor      # int32   [E + 1], as the grouped calls take them
    tokens: torch.Tensor       # int32   [T * k], the token of each row, -1: none
    slots: torch.Tensor        # int32   [T, k], the row of each choice, -1: none

    @property
    def num_experts(self) -> int:
        return self.offsets.numel() - 1

    @property
    def top_k(self) -> int:
        return self.slots.shape[1]


def _flag(value, names, what: str) -> bool:
    if not isinstance(value, str) or value not in names:
        raise ValueError(f"{what} must be one of {sorted(names)}, got {value!r}")
    return names[value]


def nf4_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
              groups: int = 1, top_groups: int = 1, group_score: str = "max", renormalize: bool = False,
              scale: float = 1.0) -> NF4Routing:
    """The top_k of the E experts of each row of logits [T, E], their weights and
    the plan.  Scores are the softmax or the sigmoid of the logits.  `bias` (float32
    [E]) moves the choice towards balance and enters no weight.  With `groups` the
    experts are chosen inside the top_groups best of so many equal runs, ranked by
    their best ("max") or their best two together ("top2").  Weights are the
    chosen scores, divided by their sum with `renormalize`, times `scale`.  An expert
    whose logit is -inf is never chosen; where fewer than top_k are left the
    places hold -1 and weight 0.  Equal scores go to the lower index."""
    return NF4Routing(*_call("route", logits, top_k, _flag(score, _SCORES, "score"), bias, groups, top_groups,
                             _flag(group_score, _GROUP_SCORES, "group_score"), renormalize, scale))


def nf4_route_bwd(grad_weights: torch.Tensor, logits: torch.Tensor, routing: NF4Routing, score: str = "softmax",
                  renormalize: bool = False, scale: float = 1.0) -> torch.Tensor:
    """grad_logits from the gradient of the weights (float32 [T, k])."""
    return _call("route_bwd", grad_weights, logits, routing.weights, routing.experts, _flag(score, _SCORES, "score"), renormalize,
                 scale)


def nf4_expert_plan(experts: torch.Tensor, E: int):
    """(offsets, tokens, slots) of a choice made elsewhere: experts int32 [T, k], an
    entry outside 0 .. E-1 being none."""
    return _call("expert_plan", experts, E)


def nf4_expert_gather(x: torch.Tensor, routing: NF4Routing, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [T, H] to the experts' rows [T * k, H].  Rows that belong to nobody are
    zeros in a result allocated here and left as they were in one passed in."""
    return _call("expert_gather", x, routing.slots, routing.offsets, out)


def nf4_expert_gather_bwd(grad_rows: torch.Tensor, routing: NF4Routing) -> torch.Tensor:
    """grad_x [T, H]: the sum of the rows of each token."""
    return _call("expert_gather_bwd", grad_rows, routing.slots)


def nf4_expert_combine(rows: torch.Tensor, routing: NF4Routing, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The experts' rows [T * k, H] back to their tokens, weighted and summed: [T, H]."""
    return _call("expert_combine", rows, routing.weights, routing.slots, routing.offsets, out)


def nf4_expert_combine_bwd(grad_out: torch.Tensor, rows: torch.Tensor, routing: NF4Routing):
    """(grad_rows [T * k, H], grad_weights float32 [T, k]); rows of nobody are zeros."""
    return _call("expert_combine_bwd", grad_out, rows, routing.weights, routing.slots, routing.offsets)
