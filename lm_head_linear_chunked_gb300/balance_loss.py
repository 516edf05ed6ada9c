"""The balance loss of a mixture of experts, with per-expert counts.

For each group of tokens (a layer, or a sequence), over the tokens that the
mask keeps: f_e is the share of the slots that name expert e, times the
number of experts, and P_e the mean router probability of e; the group's
loss is sum_e f_e P_e, 1 when the load is even.  A trainer adds it, times a
coefficient, to the head's cross-entropy:

    balance, counts = balance_loss(router_logits, experts, mask)
    loss = linear_cross_entropy(hidden, head.weight, labels) + 0.01 * balance

`balance_forward`, `balance_backward` and `balance_fused` are the library's
calls on their own; the fused one gives loss and gradient in one pass over
the logits when the coefficient is known beforehand.  The shares f take no
gradient.  There is no forward-mode derivative: a tangent is refused.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import LCEError, _flags, lce_check_status
from ._native import Traced, native


def _loss_call(router_logits, experts, mask, reduction, grad, grad_scale, grad_output, recorded=False):
    flags = _flags(reduction, False)
    r = native().balance_call(router_logits, experts, mask, bool(flags), grad, grad_scale, grad_output, recorded)
    out = {"loss": r[0], "group_loss": r[1], "counts": r[2], "n_valid": r[3], "ws": r[4]}
    if grad:
        out["grad_logits"] = r[5]
    return out


def balance_forward(router_logits: torch.Tensor, experts: torch.Tensor, mask: Optional[torch.Tensor] = None,
                    reduction: str = "mean") -> dict:
    """loss [1], group_loss [groups], counts [groups, experts], n_valid [groups] and ws (whose device status
    lce_check_status reads) of router_logits [(groups,) tokens, experts] and experts [(groups,) tokens, slots]
    (-1: an unused slot); mask [tokens] or [groups, tokens] is False where a token is left out.  The loss is the
    mean over the groups, or with reduction="sum" their sum."""
    return _loss_call(router_logits, experts, mask, reduction, False, 1.0, None)


def balance_fused(router_logits: torch.Tensor, experts: torch.Tensor, mask: Optional[torch.Tensor] = None,
                  grad_scale: float = 1.0, grad_output: Optional[torch.Tensor] = None, reduction: str = "mean") -> dict:
    """What balance_forward gives, and grad_logits: the gradient of grad_scale * grad_output * loss."""
    return _loss_call(router_logits, experts, mask, reduction, True, grad_scale, grad_output)


def balance_backward(router_logits: torch.Tensor, counts: torch.Tensor, n_valid: torch.Tensor, slots: int,
                     mask: Optional[torch.Tensor] = None, grad_scale: float = 1.0,
                     grad_output: Optional[torch.Tensor] = None, reduction: str = "mean") -> dict:
    """{"grad_logits"} of grad_scale * grad_output * loss from a forward's counts and n_valid."""
    flags = _flags(reduction, False)
    return {"grad_logits": native().balance_backward(router_logits, counts, n_valid, slots, mask, bool(flags), grad_scale,
                                                     grad_output)}


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, router_logits, experts, mask, reduction):
        out = _loss_call(router_logits, experts, mask, reduction, False, 1.0, None, True)
        ctx.save_for_backward(router_logits, mask, out["counts"], out["n_valid"])
        ctx.slots, ctx.reduction = experts.shape[-1], reduction
        ctx.mark_non_differentiable(out["counts"], out["ws"])
        return out["loss"].reshape(()), out["counts"], out["ws"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, _counts, _ws):
        router_logits, mask, counts, n_valid = ctx.saved_tensors
        g = grad_loss.reshape(1).to(torch.float32)
        d = balance_backward(router_logits, counts, n_valid, ctx.slots, mask, 1.0, g, ctx.reduction)
        return d["grad_logits"], None, None, None


def _loss(router_logits, experts, mask, reduction):
    out = balance_forward(router_logits, experts, mask, reduction)
    return out["loss"].reshape(()), out["counts"], out["ws"]


def balance_loss(router_logits: torch.Tensor, experts: torch.Tensor, mask: Optional[torch.Tensor] = None,
                 reduction: str = "mean", check: bool = False):
    """(loss, counts): the balance loss, differentiable in router_logits, and the int64 counts
    [(groups,) experts].  Arguments as balance_forward's.  check=True synchronises and raises on an expert index
    outside [-1, experts); without it such an index makes the loss NaN.  torch.jit.trace records it
    as one call."""
    call = _BalanceLoss.apply if torch.is_grad_enabled() and router_logits.requires_grad else _loss
    try:
        loss, counts, ws = call(router_logits, experts, mask, reduction)
    except Traced:
        loss, counts, ws = _BalanceLoss.apply(router_logits, experts, mask, reduction)
    if check:
        st = lce_check_status(ws, torch.cuda.current_stream(ws.device))
        if st != 0:
            raise LCEError(st, "balance loss")
    return loss, counts
