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
gradient.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import LCEError, _flags, lce_check_status
from ._tensors import address, balance_workspace, call, check_cuda, check_shape, dtype_code, stream_handle


def _shapes(logits: torch.Tensor, mask):
    """(groups, tokens, experts, type code, logits with rows in place, group stride, token stride, mask, mask
    group stride)."""
    code = dtype_code(logits, "router_logits")
    dim, shape = logits.dim(), logits.shape
    if dim not in (2, 3):
        raise ValueError(f"router_logits must be [tokens, experts] or [groups, tokens, experts], got {list(shape)}")
    T, E = shape[-2], shape[-1]
    G = shape[0] if dim == 3 else 1
    if not (G and T and E):
        raise ValueError(f"router_logits is empty: {list(shape)}")
    if logits.is_contiguous():
        zg, zt = T * E, E
    else:
        if logits.stride(-1) != 1 or (T > 1 and logits.stride(-2) < E):
            logits = logits.contiguous()
        zg = logits.stride(0) if dim == 3 else 0
        zt = logits.stride(-2) if T > 1 else E
    mg = 0
    if mask is not None:
        if mask.dtype != torch.bool:
            raise TypeError(f"mask must be bool, got {mask.dtype}")
        if mask.dim() == 2 and dim == 3:
            check_shape(mask, (G, T), "mask")
            mg = T
        else:
            check_shape(mask, (T,), "mask")
        if not mask.is_contiguous():
            mask = mask.contiguous()
    return G, T, E, code, logits, zg, zt, mask, mg


def _check_grad_output(grad_output, dev):
    if grad_output is not None:
        if grad_output.numel() != 1 or grad_output.dtype != torch.float32:
            raise TypeError("grad_output must be one float32 value")
        check_cuda(dev, grad_output)


def _loss_call(router_logits, experts, mask, reduction, stream, grad, grad_scale, grad_output):
    flags = _flags(reduction, False)
    G, T, E, code, z, zg, zt, mask, mg = _shapes(router_logits, mask)
    if experts.dtype == torch.int64:
        index_bytes = 8
    elif experts.dtype == torch.int32:
        index_bytes = 4
    else:
        raise TypeError(f"experts must be int32 or int64, got {experts.dtype}")
    lead = router_logits.shape[:-1]
    if experts.shape[:-1] != lead or experts.shape[-1] == 0:
        raise ValueError(f"experts must have shape {list(lead)} + [slots], got {list(experts.shape)}")
    if not experts.is_contiguous():
        experts = experts.contiguous()
    k = experts.shape[-1]
    dev = z.device
    check_cuda(dev, experts, mask)
    _check_grad_output(grad_output, dev)
    nws = balance_workspace(G, T, E, k)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    group_loss = torch.empty(G, dtype=torch.float32, device=dev)
    counts = torch.empty(lead[:-1] + (E,), dtype=torch.int64, device=dev)
    n_valid = torch.empty(G, dtype=torch.int64, device=dev)
    ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    out = {"loss": loss, "group_loss": group_loss, "counts": counts, "n_valid": n_valid, "ws": ws}
    if grad:
        out["grad_logits"] = dz = torch.empty_like(z, memory_format=torch.contiguous_format)
        call("lce_balance_fused", G, T, E, k, code, z.data_ptr(), zg, zt, experts.data_ptr(), index_bytes,
             address(mask), mg, grad_scale, address(grad_output), loss.data_ptr(), group_loss.data_ptr(),
             counts.data_ptr(), n_valid.data_ptr(), dz.data_ptr(), ws.data_ptr(), nws, stream_handle(stream, dev), flags)
    else:
        call("lce_balance_forward", G, T, E, k, code, z.data_ptr(), zg, zt, experts.data_ptr(), index_bytes,
             address(mask), mg, loss.data_ptr(), group_loss.data_ptr(), counts.data_ptr(), n_valid.data_ptr(),
             ws.data_ptr(), nws, stream_handle(stream, dev), flags)
    return out


def balance_forward(router_logits: torch.Tensor, experts: torch.Tensor, mask: Optional[torch.Tensor] = None,
                    reduction: str = "mean", stream=None) -> dict:
    """loss [1], group_loss [groups], counts [groups, experts], n_valid [groups] and ws (whose device status
    lce_check_status reads) of router_logits [(groups,) tokens, experts] and experts [(groups,) tokens, slots]
    (-1: an unused slot); mask [tokens] or [groups, tokens] is False where a token is left out.  The loss is the
    mean over the groups, or with reduction="sum" their sum."""
    return _loss_call(router_logits, experts, mask, reduction, stream, False, 1.0, None)


def balance_fused(router_logits: torch.Tensor, experts: torch.Tensor, mask: Optional[torch.Tensor] = None,
                  grad_scale: float = 1.0, grad_output: Optional[torch.Tensor] = None, reduction: str = "mean",
                  stream=None) -> dict:
    """What balance_forward gives, and grad_logits: the gradient of grad_scale * grad_output * loss."""
    return _loss_call(router_logits, experts, mask, reduction, stream, True, grad_scale, grad_output)


def balance_backward(router_logits: torch.Tensor, counts: torch.Tensor, n_valid: torch.Tensor, slots: int,
                     mask: Optional[torch.Tensor] = None, grad_scale: float = 1.0,
                     grad_output: Optional[torch.Tensor] = None, reduction: str = "mean", stream=None) -> dict:
    """{"grad_logits"} of grad_scale * grad_output * loss from a forward's counts and n_valid."""
    flags = _flags(reduction, False)
    G, T, E, code, z, zg, zt, mask, mg = _shapes(router_logits, mask)
    dev = z.device
    check_shape(counts, tuple(router_logits.shape[:-2]) + (E,), "counts")
    check_shape(n_valid, (G,), "n_valid")
    for what, t in (("counts", counts), ("n_valid", n_valid)):
        if t.dtype != torch.int64 or not t.is_contiguous():
            raise TypeError(f"{what} must be a contiguous int64 tensor")
    check_cuda(dev, counts, n_valid, mask)
    _check_grad_output(grad_output, dev)
    grad = torch.empty_like(z, memory_format=torch.contiguous_format)
    call("lce_balance_backward", G, T, E, slots, code, z.data_ptr(), zg, zt, counts.data_ptr(), n_valid.data_ptr(),
         address(mask), mg, grad_scale, address(grad_output), grad.data_ptr(), stream_handle(stream, dev), flags)
    return {"grad_logits": grad}


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, router_logits, experts, mask, reduction):
        out = balance_forward(router_logits, experts, mask, reduction)
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


def balance_loss(router_logits: torch.Tensor, experts: torch.Tensor, mask: Optional[torch.Tensor] = None,
                 reduction: str = "mean", check: bool = False):
    """(loss, counts): the balance loss, differentiable in router_logits, and the int64 counts
    [(groups,) experts].  Arguments as balance_forward's.  check=True synchronises and raises on an expert index
    outside [-1, experts); without it such an index makes the loss NaN."""
    if torch.is_grad_enabled() and router_logits.requires_grad:
        loss, counts, ws = _BalanceLoss.apply(router_logits, experts, mask, reduction)
    else:
        out = balance_forward(router_logits, experts, mask, reduction)
        loss, counts, ws = out["loss"].reshape(()), out["counts"], out["ws"]
    if check:
        st = lce_check_status(ws, torch.cuda.current_stream(ws.device))
        if st != 0:
            raise LCEError(st, "balance loss")
    return loss, counts
