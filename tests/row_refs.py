"""Plain float64 references of the operators between token ids and the head."""
from __future__ import annotations

import torch

from tests.op_util import U32, half_step, tiny


def rms_ref(s, weight, eps):
    """(y, rstd) of rows s."""
    s = s.double()
    rstd = (s.square().mean(-1) + eps).rsqrt()
    y = s * rstd[..., None]
    return (y if weight is None else y * weight.double()), rstd


def rms_backward_ref(dy, s, weight, rstd, ds):
    """(grad of s, grad of weight) from 2-D rows and their rstd."""
    dy, s, rstd = dy.double(), s.double(), rstd.double()[:, None]
    xh = s * rstd
    g = dy if weight is None else dy * weight.double()
    dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx if ds is None else dx + ds.double(), (dy * xh).sum(0)


def sum_depth(H: int) -> float:
    """FP32 additions that a column's term passes through in a sum over a row: what a thread adds up by itself (at
    most 64 values where rows stay in registers, H / 512 where a block reads them again), then a tree over the block."""
    return max(64.0, H / 512) + 16


def rms_tolerance(ref, H: int, dtype):
    """Of y and the like: the mean of the squares, all positive, is off by the depth of its sum, its root by half of that;
    the root's instruction by two units (4 U32), and three products follow."""
    return ref.abs() * (half_step(dtype) + (sum_depth(H) / 2 + 8) * U32) + tiny(dtype)


def embedding_grad_ref(dy, tokens, V, scale, padding=None):
    """(the gradient, the sum of magnitudes, the rows per token) in float64."""
    t, d = tokens.reshape(-1), dy.reshape(-1, dy.shape[-1]).double()
    keep = (t >= 0) & (t < V)
    if padding is not None:
        keep &= t != padding
    t, d = t[keep].long(), d[keep] * scale
    out = torch.zeros(V, d.shape[1], dtype=torch.float64, device=dy.device)
    return (out.index_add(0, t, d), out.index_add(0, t, d.abs()),
            torch.zeros(V, dtype=torch.float64, device=dy.device).index_add(0, t, torch.ones_like(t, dtype=torch.float64)))


def plan_ref(experts, E, mask, align):
    """positions, slots, counts, offsets as nested Python loops give them."""
    T, k = experts.shape
    names = experts.tolist()
    keep = [True] * T if mask is None else mask.tolist()
    R = -(-(T * k + E * (align - 1)) // align) * align
    positions, slots, counts, offsets = [[-1] * k for _ in range(T)], [-1] * R, [0] * E, [0]
    of = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if keep[t] and 0 <= names[t][j] < E:
                of[names[t][j]].append((t, j))
    at = 0
    for e in range(E):
        counts[e] = len(of[e])
        for n, (t, j) in enumerate(of[e]):
            positions[t][j] = at + n
            slots[at + n] = t * k + j
        at += -(-len(of[e]) // align) * align
        offsets.append(at)
    return (torch.tensor(positions, dtype=torch.int32).reshape(T, k), torch.tensor(slots, dtype=torch.int32),
            torch.tensor(counts), torch.tensor(offsets))
