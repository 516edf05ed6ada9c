"""Argument checks shared by the operators beside the head (layer_norm.py,
balance_loss.py, beam.py): everything that a kernel would otherwise read
through a wrong pointer, stride or type is refused here, before the call.
A small call is bound by the host, so these stay short."""
from __future__ import annotations

from functools import lru_cache

import torch

from . import BF16, F16, F32, LCEError, lce_balance_workspace_size, lce_beam_workspace_size, \
    lce_layer_norm_workspace_size, lib

DTYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}

# Workspace sizes depend on the sizes alone.
norm_workspace = lru_cache(maxsize=1024)(lce_layer_norm_workspace_size)
balance_workspace = lru_cache(maxsize=1024)(lce_balance_workspace_size)
beam_workspace = lru_cache(maxsize=1024)(lce_beam_workspace_size)


def call(name: str, *args) -> None:
    """One call of the C ABI with addresses and numbers; raises LCEError on a status other than LCE_OK."""
    status = getattr(lib(), name)(*args)
    if status:
        raise LCEError(status, name)


def dtype_code(t: torch.Tensor, what: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def check_cuda(device: torch.device, *tensors) -> None:
    """`device` is a CUDA device, and every given tensor (or None) lies on it."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {device}")
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"a tensor is on {t.device}, expected {device}")


def check_shape(t: torch.Tensor, shape: tuple, what: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {list(shape)}, got {list(t.shape)}")


def stream_handle(stream, device: torch.device) -> int:
    """The handle of `stream` (a torch.cuda.Stream, a handle, or None: the current one)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def address(t) -> int:
    """A tensor's address; None for none."""
    return None if t is None else t.data_ptr()


def rows_of(t: torch.Tensor):
    """(tensor, row stride) of t seen as rows of its last dimension: t itself
    where its rows are contiguous and evenly spaced, else a contiguous copy."""
    width = t.shape[-1]
    if t.is_contiguous():
        return t, width
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= width:
        return t, t.stride(0)
    return t.contiguous(), width
