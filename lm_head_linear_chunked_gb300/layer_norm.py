"""Layer norm in front of the LM head, with autograd.

    y = (x - mean) * rstd * weight + bias,   over the last dimension

`layer_norm` is the differentiable call and `LayerNorm` its module;
`layer_norm_forward` and `layer_norm_backward` are the two passes on their
own (one lce_layer_norm_forward or lce_layer_norm_backward call each; torch
only allocates the outputs).  x is bfloat16, float16 or float32 with any
number of leading dimensions; weight and bias are of x's type or float32,
and each may be None.  Sums are float32 in an order fixed by the sizes,
types, strides, alignment and device, so equal calls give equal bits.  There is no forward-mode derivative: a tangent is refused.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._native import Traced, native


def layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                       eps: float = 1e-5, stats: bool = True) -> dict:
    """{"y", "mean", "rstd"}: the output and, with `stats`, each row's float32
    mean and reciprocal standard deviation [number of rows], which the
    backward reads."""
    y, mean, rstd = native().norm_forward(x, weight, bias, eps, stats, False)
    return {"y": y, "mean": mean, "rstd": rstd}


def layer_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, want_grad_x: bool = True, want_grad_weight: bool = True,
                        want_grad_bias: bool = True, grad_dtype: Optional[torch.dtype] = None) -> dict:
    """{"grad_x", "grad_weight", "grad_bias"} (None where not wanted) from a
    forward's mean and rstd.  The sums over the rows are of weight's type
    (`grad_dtype`, or x's type, without a weight)."""
    dx, dw, db = native().norm_backward(grad_y, x, weight, mean, rstd, want_grad_x, want_grad_weight, want_grad_bias,
                                        grad_dtype)
    return {"grad_x": dx, "grad_weight": dw, "grad_bias": db}


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = native().norm_forward(x, weight, bias, eps, True, True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = bias.dtype if bias is not None else None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        return (*native().norm_backward(grad_y, x, weight, mean, rstd, need_x, need_w, need_b, ctx.bias_dtype), None)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Layer norm of x over its last dimension, differentiable in x, weight and bias.  torch.jit.trace records it
    as one call."""
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (bias is not None and bias.requires_grad)):
        return _LayerNorm.apply(x, weight, bias, eps)
    try:
        return native().norm_forward(x, weight, bias, eps, False, False)[0]
    except Traced:
        return _LayerNorm.apply(x, weight, bias, eps)


class LayerNorm(torch.nn.Module):
    """A layer norm with a learned weight (and bias), in place of torch.nn.LayerNorm(hidden)."""

    def __init__(self, hidden: int, eps: float = 1e-5, bias: bool = True, device=None, dtype=None):
        super().__init__()
        if hidden <= 0:
            raise ValueError("hidden must be positive")
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(hidden, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(hidden, device=device, dtype=dtype)) if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return layer_norm(x, self.weight, self.bias, self.eps)
