"""Embedding lookup with scaling, and its gradient, also into the accumulator of a tied head.

    y = scale * weight[tokens]

`embedding` is the differentiable call and `Embedding` its module; `embedding_backward` is the gradient on its own.  It
sorts the tokens and adds the rows of each in a fixed order, in float32, so equal calls give equal bits however often a
token occurs.  With a head that shares the matrix, the lookup's part is added to what the head's backward has left:

    out = fused(hidden, weight, None, labels)                                   # grad_W_acc [V, H] float32
    embedding_backward(grad_h, tokens, V, out=out["grad_W_acc"], accumulate=True)

tokens are int32 or int64 of any shape, weight [V, H] is bfloat16, float16 or float32.  A token equal to `padding_idx`
gets no gradient; its y is its row, or zero where padding_idx lies outside [0, V) (such as -1).  Another token outside
[0, V) gives a row of NaN, and with check=True an error.  There is no forward-mode derivative: a tangent is refused.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import LCEError, lce_check_status
from ._native import Traced, native


def _raise_on(word, where: str) -> None:
    status = lce_check_status(word, torch.cuda.current_stream(word.device))
    if status != 0:
        raise LCEError(status, where)


def embedding_backward(grad_y: torch.Tensor, tokens: torch.Tensor, vocab: int, scale: float = 1.0,
                       padding_idx: Optional[int] = None, dtype: Optional[torch.dtype] = None,
                       out: Optional[torch.Tensor] = None, accumulate: bool = False, check: bool = False) -> torch.Tensor:
    """grad_weight [vocab, H] from grad_y [..., H]: of grad_y's type, or float32 as `dtype` or `out` say.  `out` is
    written (all of it: zeros where no token names a row) and returned; with accumulate=True it is float32 and added
    to, and rows that no token names are left alone.  check=True synchronises and raises on a token outside the
    vocabulary."""
    grad, ws = native().embedding_backward(grad_y, tokens, vocab, scale, padding_idx, dtype, out, accumulate)
    if check:
        _raise_on(ws, "embedding_backward")
    return grad


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, tokens, scale, padding_idx, status):
        ctx.save_for_backward(tokens)
        ctx.vocab, ctx.scale, ctx.padding_idx = weight.shape[0], scale, padding_idx
        return native().embedding_forward(tokens, weight, scale, padding_idx, status, True)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        tokens, = ctx.saved_tensors
        grad, _ = native().embedding_backward(grad_y, tokens, ctx.vocab, ctx.scale, ctx.padding_idx, None, None, False)
        return grad, None, None, None, None


def embedding(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0, padding_idx: Optional[int] = None,
              check: bool = False) -> torch.Tensor:
    """scale * weight[tokens], [..., H] of weight's type, differentiable in weight.  check=True synchronises and raises
    on a token outside the vocabulary.  torch.jit.trace records it as one call."""
    status = torch.zeros(64, dtype=torch.int32, device=weight.device) if check else None
    if torch.is_grad_enabled() and weight.requires_grad:
        y = _Embedding.apply(weight, tokens, scale, padding_idx, status)
    else:
        try:
            y = native().embedding_forward(tokens, weight, scale, padding_idx, status, False)
        except Traced:
            y = _Embedding.apply(weight, tokens, scale, padding_idx, status)
    if check:
        _raise_on(status, "embedding")
    return y


class Embedding(torch.nn.Module):
    """A learned embedding, in place of torch.nn.Embedding(vocab, hidden); `scale` multiplies what is looked up.  Its
    weight may be a head's (head.weight = embedding.weight)."""

    def __init__(self, vocab: int, hidden: int, scale: float = 1.0, padding_idx: Optional[int] = None, device=None,
                 dtype=None):
        super().__init__()
        if vocab <= 0 or hidden <= 0:
            raise ValueError("vocab and hidden must be positive")
        self.scale, self.padding_idx = scale, padding_idx
        self.weight = torch.nn.Parameter(torch.randn(vocab, hidden, device=device, dtype=dtype))
        if padding_idx is not None and 0 <= padding_idx < vocab:
            with torch.no_grad():
                self.weight[padding_idx].zero_()

    def forward(self, tokens: torch.Tensor) -> torch.Tensor:
        return embedding(tokens, self.weight, self.scale, self.padding_idx)
