"""Helpers of the tests of the operators beside the head (layer norm, balance
loss, beam selection)."""
from __future__ import annotations

import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U32 = 2.0 ** -24  # half a step of fp32


def half_step(dtype: torch.dtype) -> float:
    """The largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype: torch.dtype) -> float:
    """Half the spacing of the type's subnormals: the absolute error of rounding a value near zero."""
    i = torch.finfo(dtype)
    return i.smallest_normal * i.eps / 2


def assert_within(got: torch.Tensor, ref: torch.Tensor, tol: torch.Tensor, what: str) -> None:
    """|got - ref| <= tol element by element, in float64; ref is finite."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    d = (got.detach().double() - ref).abs()
    bad = ~(d <= tol)
    if bool(bad.any()):
        i = tuple(int(k) for k in bad.nonzero()[0])
        t = tol if tol.dim() == 0 else tol.expand_as(d)[i]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; at {i}: got {got[i].item():.9g}, "
                             f"expected {ref[i].item():.9g}, allowed {float(t):.3g}")


def normal(shape, seed, dtype=torch.float32, std=1.0, mean=0.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.empty(shape, dtype=torch.float32, device=device).normal_(mean, std, generator=g).to(dtype)
