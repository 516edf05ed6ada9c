"""RMS norm with the residual's addition in front of it, with autograd and with an output in 8 bits.

    s = x + residual, rounded to their type        (x itself without a residual)
    y = s * rstd * weight,   rstd = 1 / sqrt(mean(s^2) + eps),   over the last dimension

A block of a model adds its output to the residual and norms the sum for the next one:

    h, residual = rms_norm(block(h), weight, residual)

`rms_norm` is the differentiable call and `RMSNorm` its module; `rms_norm_forward` and `rms_norm_backward` are the two
passes on their own, `rms_norm_fp8` the forward with its output in e4m3 and scales, in front of 8-bit products (one call
of the library each; torch only allocates the outputs).  x is bfloat16, float16 or float32 with any number of leading
dimensions; weight is of x's type or float32, and may be None.  Sums are float32 in an order fixed by the sizes, types,
strides, alignment and device, so equal calls give equal bits.  There is no forward-mode derivative: a tangent is refused.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import FP8_GROUP
from ._native import Traced, native


def rms_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                     eps: float = 1e-6, stats: bool = True) -> dict:
    """{"y", "sum", "rstd"}: the output; what was normed (x itself without a residual); and, with `stats`, each row's
    float32 reciprocal root mean square [number of rows], which the backward reads."""
    y, total, rstd = native().rms_forward(x, weight, residual, eps, stats, False)
    return {"y": y, "sum": x if total is None else total, "rstd": rstd}


def rms_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor,
                      grad_sum: Optional[torch.Tensor] = None, want_grad_x: bool = True,
                      want_grad_weight: bool = True) -> dict:
    """{"grad_x", "grad_weight"} (None where not wanted, grad_weight also without a weight) from a forward's "sum" as x
    and its rstd.  grad_x is the gradient of x and of the residual alike; grad_sum is added to it (what arrives at the
    sum from behind the norm)."""
    dx, dw = native().rms_backward(grad_y, x, weight, rstd, grad_sum, want_grad_x, want_grad_weight)
    return {"grad_x": dx, "grad_weight": dw}


def rms_norm_fp8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, group: int = FP8_GROUP) -> dict:
    """{"q", "scales", "sum"}: the output as float8_e4m3fn q (x's shape) and float32 scales [..., groups], y being about
    q * scale: one scale for every `group` = 128 columns (the last group may be shorter), or with group=0 one for the
    row.  A scale is the largest magnitude / 448, q the rounded y * (1 / scale).  Not differentiable."""
    q, scales, total = native().rms_fp8(x, weight, residual, eps, group)
    return {"q": q, "scales": scales, "sum": x if total is None else total}


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, total, rstd = native().rms_forward(x, weight, residual, eps, True, True)
        ctx.save_for_backward(x if total is None else total, weight, rstd)
        ctx.set_materialize_grads(False)
        return y if total is None else (y, total)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y, grad_sum=None):
        x, weight, rstd = ctx.saved_tensors
        need_x, need_w, need_r, _ = ctx.needs_input_grad
        if grad_y is None:  # only the sum is used
            return grad_sum if need_x else None, None, grad_sum if need_r else None, None
        dx, dw = native().rms_backward(grad_y, x, weight, rstd, grad_sum, need_x or need_r, need_w)
        return dx if need_x else None, dw, dx if need_r else None, None


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6):
    """y, or with a residual (y, sum): the RMS norm of x + residual over the last dimension, and the sum.
    Differentiable in x, weight and residual.  torch.jit.trace records it as one call."""
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (residual is not None and residual.requires_grad)):
        return _RmsNorm.apply(x, weight, residual, eps)
    try:
        y, total, _ = native().rms_forward(x, weight, residual, eps, False, False)
    except Traced:
        return _RmsNorm.apply(x, weight, residual, eps)
    return y if total is None else (y, total)


class RMSNorm(torch.nn.Module):
    """An RMS norm with a learned weight, in place of torch.nn.RMSNorm(hidden); called with a residual it also adds it
    and returns (y, sum)."""

    def __init__(self, hidden: int, eps: float = 1e-6, device=None, dtype=None):
        super().__init__()
        if hidden <= 0:
            raise ValueError("hidden must be positive")
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(hidden, device=device, dtype=dtype))

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        return rms_norm(x, self.weight, residual, self.eps)
