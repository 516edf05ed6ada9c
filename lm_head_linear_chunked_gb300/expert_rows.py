"""A mixture's tokens sorted by expert, and back, with autograd.

    plan = expert_plan(experts, n_experts, mask)     # experts [tokens, slots], as balance_loss takes them
    rows = dispatch(x, plan)                         # each expert's tokens side by side
    out = products(rows, plan["offsets"])            # the experts' own work, on rows offsets[e] .. offsets[e + 1]
    y = combine(out, weights, plan)                  # sum over a token's slots of weights * out

A slot's row holds its token's x; expert e's rows lie in the order of tokens and slots.  With `align` every segment
starts on a multiple of it (the tiles of a grouped product), and rows that no slot takes are zero, in dispatch and in the
gradient of combine's rows.  `dispatch` and `combine` are differentiable; `dispatch_backward`, `combine_backward` are
their gradients on their own.  Sums are float32 in a fixed order.  There is no forward-mode derivative: a tangent is
refused.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import LCEError, lce_check_status
from ._native import Traced, native


def expert_plan(experts: torch.Tensor, n_experts: int, mask: Optional[torch.Tensor] = None, align: int = 1,
                check: bool = False) -> dict:
    """Sorts the slots of experts [..., slots] (int32 or int64; -1: unused) by expert; mask [...] is False where a token
    is left out.  Returns {"positions" int32 [..., slots]: the row of each slot (-1: none); "slots" int32 [rows]: the
    number of each row's slot, token * slots + slot (-1: none); "counts" int64 [n_experts]; "offsets" int64
    [n_experts + 1]: where each expert's rows start, multiples of `align`; "ws": its device status}.  There are as many
    rows as any choice of experts can take.  Another index outside [0, n_experts) counts as unused, and check=True
    synchronises and raises on one."""
    positions, slots, counts, offsets, ws = native().expert_plan(experts, n_experts, mask, align)
    if check:
        status = lce_check_status(ws, torch.cuda.current_stream(ws.device))
        if status != 0:
            raise LCEError(status, "expert_plan")
    return {"positions": positions, "slots": slots, "counts": counts, "offsets": offsets, "ws": ws}


def dispatch_backward(grad_rows: torch.Tensor, plan: dict) -> torch.Tensor:
    """grad_x [..., H]: the sum over each token's slots of grad_rows [rows, H]."""
    return native().expert_dispatch_backward(grad_rows, plan["positions"], plan["slots"])


def combine_backward(grad_y: torch.Tensor, rows: torch.Tensor, weights: Optional[torch.Tensor], plan: dict,
                     want_grad_rows: bool = True, want_grad_weights: bool = True) -> dict:
    """{"grad_rows", "grad_weights"} (None where not wanted, grad_weights also without weights) of combine."""
    dr, dw = native().expert_combine_backward(grad_y, rows, weights, plan["positions"], plan["slots"], want_grad_rows,
                                              want_grad_weights)
    return {"grad_rows": dr, "grad_weights": dw}


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, slots):
        ctx.save_for_backward(positions, slots)
        return native().expert_dispatch(x, positions, slots, True)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_rows):
        return native().expert_dispatch_backward(grad_rows, *ctx.saved_tensors), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, positions, slots):
        ctx.save_for_backward(rows, weights, positions, slots)
        return native().expert_combine(rows, weights, positions, slots, True)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        rows, weights, positions, slots = ctx.saved_tensors
        need_rows, need_weights = ctx.needs_input_grad[:2]
        dr, dw = native().expert_combine_backward(grad_y, rows, weights, positions, slots, need_rows, need_weights)
        return dr, dw, None, None


def dispatch(x: torch.Tensor, plan: dict) -> torch.Tensor:
    """rows [rows, H]: x [..., H] by the plan of its tokens' experts, zero where no slot takes a row.  Differentiable in
    x.  torch.jit.trace records it as one call."""
    positions, slots = plan["positions"], plan["slots"]
    if torch.is_grad_enabled() and x.requires_grad:
        return _Dispatch.apply(x, positions, slots)
    try:
        return native().expert_dispatch(x, positions, slots, False)
    except Traced:
        return _Dispatch.apply(x, positions, slots)


def combine(rows: torch.Tensor, weights: Optional[torch.Tensor], plan: dict) -> torch.Tensor:
    """y [..., H]: for each token the sum over its slots of weights [..., slots] (of rows' type or float32; None: 1)
    times their rows.  Differentiable in rows and weights.  torch.jit.trace records it as one call."""
    positions, slots = plan["positions"], plan["slots"]
    if torch.is_grad_enabled() and (rows.requires_grad or (weights is not None and weights.requires_grad)):
        return _Combine.apply(rows, weights, positions, slots)
    try:
        return native().expert_combine(rows, weights, positions, slots, False)
    except Traced:
        return _Combine.apply(rows, weights, positions, slots)
