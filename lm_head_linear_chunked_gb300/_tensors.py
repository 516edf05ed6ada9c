"""Argument checks shared by the operators beside the head (layer_norm.py,
balance_loss.py, beam.py): everything that a kernel would otherwise read
through a wrong pointer, stride or type is refused here, before the call."""
from __future__ import annotations

import torch

from . import BF16, F16, F32

DTYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}


def dtype_code(t: torch.Tensor, what: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def check_cuda(device: torch.device, **tensors) -> None:
    """Every given tensor lies on the CUDA device `device`."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {device}")
    for what, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{what} is on {t.device}, expected {device}")


def check_shape(t: torch.Tensor, shape: tuple, what: str) -> None:
    if tuple(t.shape) != shape:
        raise ValueError(f"{what} must have shape {list(shape)}, got {list(t.shape)}")


def rows_of(t: torch.Tensor):
    """(tensor, row stride) of t seen as rows of its last dimension: t itself
    where its rows are contiguous and evenly spaced, else a contiguous copy."""
    width = t.shape[-1]
    if t.is_contiguous():
        return t, width
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= width:
        return t, t.stride(0)
    return t.contiguous(), width
