"""Beam search over the LM head's logits: the selection, and the states.

    logits = model(tokens[:, -1:], caches)                       # [items, beams, V]
    step = beam_select(logits, scores, eos_token=eos)
    caches = beam_reorder(caches, step["parents"], out=other)    # a second set of buffers
    scores, token, finished = step["scores"], step["tokens"], step["finished"]

`beam_select` is one lce_beam_select call (two kernels: a scan of the
vocabulary and the joining of its parts), `beam_reorder` one
lce_beam_reorder call for all states; torch only allocates the outputs.
Neither is differentiable; a forward-mode tangent and torch.jit.trace are
refused.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import LCEError, lce_check_status
from ._native import native


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n: Optional[int] = None,
                finished: Optional[torch.Tensor] = None, pad_token: int = 0, eos_token: Optional[int] = None) -> dict:
    """The n (default: beams) best continuations of each item.

    logits [items, beams, V] (bfloat16, float16 or float32), scores [items, beams] float32 (a beam with -inf
    is dead, as all but the first are before the first step), finished [items, beams] bool: such a beam goes on
    as itself, with pad_token and its score.  Returns {"scores" float32, "tokens" int64, "parents" int64 (the
    beam)}, each [items, n], best first; equal scores go to the lower beam, then the larger logit, then the
    lower token.  With eos_token also "finished" [items, n]: the parent was finished or the token is
    eos_token."""
    n = (logits.shape[1] if logits.dim() == 3 else 0) if n is None else n
    if n <= 0 and logits.dim() == 3 and logits.numel():
        raise ValueError("n must be positive")
    if eos_token is not None and eos_token < 0:
        raise ValueError("eos_token must not be negative")
    r = native().beam_select(logits, scores, n, finished, pad_token, -1 if eos_token is None else eos_token)
    out = {"scores": r[0], "tokens": r[1], "parents": r[2]}
    if eos_token is not None:
        out["finished"] = r[3]
    return out


def beam_reorder(states: Sequence[torch.Tensor], parents: torch.Tensor,
                 out: Optional[Sequence[torch.Tensor]] = None, check: bool = False) -> list:
    """Moves the beams' states to where the selection wants them.

    states: tensors [items * beams, ...] of any type (caches, token histories); parents [items, n] int64, each
    row's beams by their index within the item.  Returns tensors [items * n, ...] whose row item * n + j is row
    item * beams + parents[item, j] of the state.  `out` gives the buffers (such as a second set of caches, or
    views of their used part: strides are kept, and only the elements of the views move); they must not overlap
    the states, each other or themselves.  A parent outside [0, beams) gives a row of zeros; check=True synchronises and raises on one."""
    status = torch.zeros(64, dtype=torch.int32, device=parents.device) if check else None
    out = native().beam_reorder(list(states), parents, None if out is None else list(out), status)
    if check and out:
        st = lce_check_status(status, torch.cuda.current_stream(parents.device))
        if st != 0:
            raise LCEError(st, "beam_reorder")
    return out
