"""Beam search over the LM head's logits: the selection, and the states.

    logits = model(tokens[:, -1:], caches)                       # [items, beams, V]
    step = beam_select(logits, scores, eos_token=eos)
    caches = beam_reorder(caches, step["parents"], out=other)    # a second set of buffers
    scores, token, finished = step["scores"], step["tokens"], step["finished"]

`beam_select` is one lce_beam_select call (two kernels: a scan of the
vocabulary and the joining of its parts), `beam_reorder` one
lce_beam_reorder call for all states; torch only allocates the outputs.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import Optional, Sequence

import torch

from . import BeamState, LCEError, lce_check_status
from ._tensors import address, beam_workspace, call, check_cuda, check_shape, dtype_code, stream_handle


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n: Optional[int] = None,
                finished: Optional[torch.Tensor] = None, pad_token: int = 0, eos_token: Optional[int] = None,
                stream=None) -> dict:
    """The n (default: beams) best continuations of each item.

    logits [items, beams, V] (bfloat16, float16 or float32), scores [items, beams] float32 (a beam with -inf
    is dead, as all but the first are before the first step), finished [items, beams] bool: such a beam goes on
    as itself, with pad_token and its score.  Returns {"scores" float32, "tokens" int64, "parents" int64 (the
    beam)}, each [items, n], best first; equal scores go to the lower beam, then the larger logit, then the
    lower token.  With eos_token also "finished" [items, n]: the parent was finished or the token is
    eos_token."""
    code = dtype_code(logits, "logits")
    if logits.dim() != 3 or 0 in logits.shape:
        raise ValueError(f"logits must be [items, beams, V] and not empty, got {list(logits.shape)}")
    B, K, V = logits.shape
    check_shape(scores, (B, K), "scores")
    if scores.dtype != torch.float32:
        raise TypeError(f"scores must be float32, got {scores.dtype}")
    if finished is not None:
        check_shape(finished, (B, K), "finished")
        if finished.dtype != torch.bool:
            raise TypeError(f"finished must be bool, got {finished.dtype}")
        finished = finished.contiguous()
    n = K if n is None else n
    if n <= 0:
        raise ValueError("n must be positive")
    if eos_token is not None and eos_token < 0:
        raise ValueError("eos_token must not be negative")
    dev = logits.device
    check_cuda(dev, scores, finished)
    # rows evenly spaced (as a last position's logits are in [items * beams, length, V])?
    ld = V
    if not logits.is_contiguous():
        ld = logits.stride(1) if K > 1 else logits.stride(0) if B > 1 else V
        if logits.stride(2) != 1 or ld < V or (B > 1 and K > 1 and logits.stride(0) != K * ld):
            logits, ld = logits.contiguous(), V
    if not scores.is_contiguous():
        scores = scores.contiguous()
    nws = beam_workspace(B, K, V, n)
    ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    tokens = torch.empty((B, n), dtype=torch.int64, device=dev)
    parents = torch.empty_like(tokens)
    out = {"scores": torch.empty((B, n), dtype=torch.float32, device=dev), "tokens": tokens, "parents": parents}
    ended = None
    if eos_token is None:
        eos_token = -1
    else:
        out["finished"] = ended = torch.empty((B, n), dtype=torch.bool, device=dev)
    call("lce_beam_select", B, K, V, n, code, logits.data_ptr(), ld, scores.data_ptr(), address(finished), pad_token,
         eos_token, out["scores"].data_ptr(), tokens.data_ptr(), parents.data_ptr(), address(ended), ws.data_ptr(),
         nws, stream_handle(stream, dev))
    return out


@lru_cache(maxsize=4096)
def _layout(shape: tuple, src: tuple, dst: tuple, size: int):
    """A state's row as the C ABI describes it, (n1, strides, n2, strides, run) in bytes, from the shape and the
    strides of src and dst; None where that takes more than two strided dimensions."""
    dims = []  # outermost first: [size, src stride, dst stride]
    for n, a, b in zip(shape[1:], src[1:], dst[1:]):
        if n == 1:
            continue
        if dims and dims[-1][1] == n * a and dims[-1][2] == n * b:
            dims[-1] = [dims[-1][0] * n, a, b]
        else:
            dims.append([n, a, b])
    run = 1
    if dims and dims[-1][1] == 1 and dims[-1][2] == 1:
        run = dims.pop()[0]
    if len(dims) > 2:
        return None
    (n1, s1, d1), (n2, s2, d2) = [[1, 0, 0]] * (2 - len(dims)) + dims
    return n1, s1 * size, d1 * size, n2, s2 * size, d2 * size, run * size


@lru_cache(maxsize=4096)
def _bytes_spanned(shape: tuple, strides: tuple, size: int) -> int:
    """Bytes from a tensor's first to its last (0 for an empty one)."""
    return 0 if 0 in shape else (sum((n - 1) * s for n, s in zip(shape, strides)) + 1) * size


def _overlap(ranges) -> bool:
    """Whether a range (first, end, whose) of one side meets one of the other's."""
    ends = [0, 0]
    for first, end, whose in sorted(ranges):
        if first < ends[1 - whose]:
            return True
        ends[whose] = max(ends[whose], end)
    return False


def beam_reorder(states: Sequence[torch.Tensor], parents: torch.Tensor,
                 out: Optional[Sequence[torch.Tensor]] = None, check: bool = False, stream=None) -> list:
    """Moves the beams' states to where the selection wants them.

    states: tensors [items * beams, ...] of any type (caches, token histories); parents [items, n] int64, each
    row's beams by their index within the item.  Returns tensors [items * n, ...] whose row item * n + j is row
    item * beams + parents[item, j] of the state.  `out` gives the buffers (such as a second set of caches, or
    views of their used part: strides are kept, and only the elements of the views move); they must not overlap
    the states.  A parent outside [0, beams) gives a row of zeros; check=True synchronises and raises on one."""
    states = list(states)
    if parents.dim() != 2 or parents.dtype != torch.int64 or 0 in parents.shape:
        raise ValueError("parents must be int64 [items, n] and not empty")
    B, n = parents.shape
    if not states:
        return []
    if states[0].dim() == 0 or states[0].shape[0] == 0 or states[0].shape[0] % B:
        raise ValueError(f"a state's first dimension must be a multiple of the {B} items")
    rows, dev = states[0].shape[0], states[0].device
    fresh = out is None
    out = [torch.empty((B * n,) + tuple(t.shape[1:]), dtype=t.dtype, device=t.device) for t in states] \
        if fresh else list(out)
    if len(out) != len(states):
        raise ValueError(f"{len(states)} states, but {len(out)} outputs")
    fields, ranges, keep = [], [], []  # keep: contiguous copies live until the launch is enqueued
    for i, (a, b) in enumerate(zip(states, out)):
        shape = tuple(a.shape)
        if not shape or shape[0] != rows:
            raise ValueError(f"states must have {rows} rows each, states[{i}] has shape {list(shape)}")
        if tuple(b.shape) != (B * n,) + shape[1:]:
            check_shape(b, (B * n,) + shape[1:], f"out[{i}]")
        if a.dtype != b.dtype:
            raise TypeError(f"out[{i}] must be {a.dtype}, got {b.dtype}")
        if b.device != dev or a.device != dev:
            raise ValueError(f"states and outputs must be on {dev}")
        size, strides, to = a.element_size(), a.stride(), b.stride()
        span = _bytes_spanned(shape, strides, size)
        if not span:
            continue
        src, dst = a.data_ptr(), b.data_ptr()
        if not fresh:
            ranges.append((src, src + span, 0))
            ranges.append((dst, dst + _bytes_spanned((B * n,) + shape[1:], to, size), 1))
        row = _layout(shape, strides, to, size)
        if row is None:
            a = a.contiguous()
            keep.append(a)
            src, strides = a.data_ptr(), a.stride()
            row = _layout(shape, strides, to, size)
            if row is None:
                raise ValueError(f"an output's strides {to} have more than two strided dimensions")
        fields += (src, dst, strides[0] * size, to[0] * size)
        fields += row
    check_cuda(dev, parents)
    if _overlap(ranges):
        raise ValueError("out overlaps the states")
    if not parents.is_contiguous():
        parents = parents.contiguous()
    array = (ctypes.c_int64 * len(fields))(*fields)
    handle = stream_handle(stream, dev)
    status = torch.zeros(64, dtype=torch.int32, device=dev) if check else None
    call("lce_beam_reorder", B, rows // B, n, parents.data_ptr(), ctypes.cast(array, ctypes.POINTER(BeamState)),
         len(fields) // 11, address(status), handle)
    if check:
        st = lce_check_status(status, handle)
        if st != 0:
            raise LCEError(st, "beam_reorder")
    return out
