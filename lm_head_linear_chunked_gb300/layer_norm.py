"""Layer norm in front of the LM head, with autograd.

    y = (x - mean) * rstd * weight + bias,   over the last dimension

`layer_norm` is the differentiable call and `LayerNorm` its module;
`layer_norm_forward` and `layer_norm_backward` are the two passes on their
own (one lce_layer_norm_forward or lce_layer_norm_backward call each; torch
only allocates the outputs).  x is bfloat16, float16 or float32 with any
number of leading dimensions; weight and bias are of x's type or float32,
and each may be None.  Sums are float32 in a fixed order, so equal calls
give equal bits.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import F32
from ._tensors import address, call, check_cuda, check_shape, dtype_code, norm_workspace, rows_of, stream_handle


def _width(x: torch.Tensor) -> int:
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x needs a last dimension of at least one element")
    return x.shape[-1]


def _check_affine(x, H, t, what):
    if t.shape != (H,):
        check_shape(t, (H,), what)
    if t.dtype != x.dtype and t.dtype != torch.float32:
        raise TypeError(f"{what} must be {x.dtype} or float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                       eps: float = 1e-5, stats: bool = True, stream=None) -> dict:
    """{"y", "mean", "rstd"}: the output and, with `stats`, each row's float32
    mean and reciprocal standard deviation [number of rows], which the
    backward reads."""
    code = wcode = dtype_code(x, "x")
    H = _width(x)
    if weight is not None:
        _check_affine(x, H, weight, "weight")
        wcode = code if weight.dtype == x.dtype else F32
    if bias is not None:
        _check_affine(x, H, bias, "bias")
        if weight is not None and weight.dtype != bias.dtype:
            raise TypeError(f"weight and bias must have one type, got {weight.dtype} and {bias.dtype}")
        wcode = code if bias.dtype == x.dtype else F32
    dev = x.device
    check_cuda(dev, weight, bias)
    x, ldx = rows_of(x)
    rows = x.numel() // H
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    mean = rstd = None
    if stats:
        mean = torch.empty(rows, dtype=torch.float32, device=dev)
        rstd = torch.empty_like(mean)
    call("lce_layer_norm_forward", rows, H, code, wcode, x.data_ptr(), ldx, address(weight), address(bias), eps,
         y.data_ptr(), H, address(mean), address(rstd), stream_handle(stream, dev))
    return {"y": y, "mean": mean, "rstd": rstd}


def layer_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, want_grad_x: bool = True, want_grad_weight: bool = True,
                        want_grad_bias: bool = True, grad_dtype: Optional[torch.dtype] = None, stream=None) -> dict:
    """{"grad_x", "grad_weight", "grad_bias"} (None where not wanted) from a
    forward's mean and rstd.  The sums over the rows are of weight's type
    (`grad_dtype`, or x's type, without a weight)."""
    code = dtype_code(x, "x")
    H = _width(x)
    if grad_y.shape != x.shape:
        check_shape(grad_y, tuple(x.shape), "grad_y")
    if grad_y.dtype != x.dtype:
        raise TypeError(f"grad_y must be {x.dtype}, got {grad_y.dtype}")
    if weight is not None:
        _check_affine(x, H, weight, "weight")
        gdtype = weight.dtype
    else:
        gdtype = grad_dtype or x.dtype
        if gdtype != x.dtype and gdtype != torch.float32:
            raise TypeError(f"grad_dtype must be {x.dtype} or float32, got {gdtype}")
    rows = x.numel() // H
    for what, t in (("mean", mean), ("rstd", rstd)):
        if t.shape != (rows,):
            check_shape(t, (rows,), what)
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise TypeError(f"{what} must be a contiguous float32 tensor")
    dev = x.device
    check_cuda(dev, grad_y, weight, mean, rstd)
    x, ldx = rows_of(x)
    grad_y, ldg = rows_of(grad_y)
    grad_x = torch.empty_like(x, memory_format=torch.contiguous_format) if want_grad_x else None
    grad_weight = grad_bias = ws = None
    nws = 0
    if want_grad_weight:
        grad_weight = torch.empty(H, dtype=gdtype, device=dev)
    if want_grad_bias:
        grad_bias = torch.empty(H, dtype=gdtype, device=dev)
    if want_grad_weight or want_grad_bias:
        nws = norm_workspace(rows, H)
        ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    if want_grad_x or ws is not None:
        call("lce_layer_norm_backward", rows, H, code, code if gdtype == x.dtype else F32, grad_y.data_ptr(), ldg,
             x.data_ptr(), ldx, address(weight), mean.data_ptr(), rstd.data_ptr(), address(grad_x), H,
             address(grad_weight), address(grad_bias), address(ws), nws, stream_handle(stream, dev))
    return {"grad_x": grad_x, "grad_weight": grad_weight, "grad_bias": grad_bias}


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        out = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, out["mean"], out["rstd"])
        ctx.bias_dtype = bias.dtype if bias is not None else None
        return out["y"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        d = layer_norm_backward(grad_y, x, weight, mean, rstd, need_x, need_w, need_b, ctx.bias_dtype)
        return d["grad_x"], d["grad_weight"], d["grad_bias"], None


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Layer norm of x over its last dimension, differentiable in x, weight and bias."""
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (bias is not None and bias.requires_grad)):
        return _LayerNorm.apply(x, weight, bias, eps)
    return layer_norm_forward(x, weight, bias, eps, stats=False)["y"]


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
