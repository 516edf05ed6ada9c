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

from typing import Optional, Sequence

import torch

from . import BeamState, LCEError, lce_beam_reorder, lce_beam_select, lce_beam_workspace_size, lce_check_status
from ._tensors import check_cuda, check_shape, dtype_code


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
    check_cuda(dev, scores=scores, finished=finished)
    # rows evenly spaced (as a last position's logits are in [items * beams, length, V])?
    ld = logits.stride(1) if K > 1 else logits.stride(0) if B > 1 else V
    if logits.stride(2) != 1 or ld < V or (B > 1 and K > 1 and logits.stride(0) != K * ld):
        logits, ld = logits.contiguous(), V
    scores = scores.contiguous()
    nws = lce_beam_workspace_size(B, K, V, n)
    ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    tokens, parents = torch.empty((2, B, n), dtype=torch.int64, device=dev).unbind(0)
    out = {"scores": torch.empty((B, n), dtype=torch.float32, device=dev), "tokens": tokens, "parents": parents}
    if eos_token is not None:
        out["finished"] = torch.empty((B, n), dtype=torch.bool, device=dev)
    lce_beam_select(B, K, V, n, code, logits, ld, scores, finished, pad_token, -1 if eos_token is None else eos_token,
                    out["scores"], tokens, parents, out.get("finished"), ws, nws,
                    stream or torch.cuda.current_stream(dev))
    return out


def _runs(src: torch.Tensor, dst: torch.Tensor):
    """A state's row as (n1, strides, n2, strides, run) in elements, the same for src and dst; None where that
    takes more than two strided dimensions."""
    dims = []  # outermost first: [size, src stride, dst stride]
    for size, a, b in zip(src.shape[1:], src.stride()[1:], dst.stride()[1:]):
        if size == 1:
            continue
        if dims and dims[-1][1] == size * a and dims[-1][2] == size * b:
            dims[-1] = [dims[-1][0] * size, a, b]
        else:
            dims.append([size, a, b])
    run = 1
    if dims and dims[-1][1] == 1 and dims[-1][2] == 1:
        run = dims.pop()[0]
    if len(dims) > 2:
        return None
    dims = [[1, 0, 0]] * (2 - len(dims)) + dims
    return dims[0], dims[1], run


def _extent(t: torch.Tensor):
    """The addresses from t's first to its last byte."""
    first = t.data_ptr()
    return first, first + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


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
    for i, (a, b) in enumerate(zip(states, out)):
        if a.dim() == 0 or a.shape[0] != rows:
            raise ValueError(f"states must have {rows} rows each, states[{i}] has shape {list(a.shape)}")
        check_shape(b, (B * n,) + tuple(a.shape[1:]), f"out[{i}]")
        if a.dtype != b.dtype:
            raise TypeError(f"out[{i}] must be {a.dtype}, got {b.dtype}")
        if b.device != dev or a.device != dev:
            raise ValueError(f"states and outputs must be on {dev}")
    check_cuda(dev, parents=parents)
    extents = [] if fresh else [_extent(b) for b in out if b.numel()]
    for lo, hi in (_extent(a) for a in states if a.numel()) if extents else ():
        if any(lo < h and l < hi for l, h in extents):
            raise ValueError("out overlaps the states")
    array = (BeamState * len(states))()
    keep = []  # contiguous copies live until the launch is enqueued
    for s, a, b in zip(array, states, out):
        if a.numel() == 0:
            continue
        r = _runs(a, b)
        if r is None:
            a = a.contiguous()
            keep.append(a)
            r = _runs(a, b)
            if r is None:
                raise ValueError(f"an output's strides {b.stride()} have more than two strided dimensions")
        (n1, s1, d1), (n2, s2, d2), run = r
        size = a.element_size()
        s.src, s.dst = a.data_ptr(), b.data_ptr()
        s.src_row, s.dst_row = a.stride(0) * size, b.stride(0) * size
        s.n1, s.src1, s.dst1 = n1, s1 * size, d1 * size
        s.n2, s.src2, s.dst2 = n2, s2 * size, d2 * size
        s.run_bytes = run * size
    stream = stream or torch.cuda.current_stream(dev)
    status = torch.zeros(64, dtype=torch.int32, device=dev) if check else None
    lce_beam_reorder(B, rows // B, n, parents.contiguous(), array, len(states), status, stream)
    if check:
        st = lce_check_status(status, stream)
        if st != 0:
            raise LCEError(st, "beam_reorder")
    return out
