"""What torch's transforms may not do with the operators beside the head,
without a GPU: their calls work on addresses, so a forward-mode tangent is
refused instead of lost, and a trace would record outputs that nothing fills."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import __graft_entry__
from lm_head_linear_chunked_gb300.balance_loss import balance_backward, balance_forward, balance_fused, balance_loss
from lm_head_linear_chunked_gb300.beam import beam_reorder, beam_select
from lm_head_linear_chunked_gb300.layer_norm import layer_norm, layer_norm_backward, layer_norm_forward


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


X, W, S = torch.zeros(4, 16), torch.ones(16), torch.zeros(4)
Z, E = torch.zeros(2, 10, 8), torch.zeros(2, 10, 2, dtype=torch.int64)
C, N, G = torch.zeros(2, 8, dtype=torch.int64), torch.zeros(2, dtype=torch.int64), torch.ones(1)
L, B, P = torch.zeros(2, 3, 20), torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int64)
T = torch.zeros(6, 5)

# each with the tensor that gets the tangent, and the call
CALLS = [
    (X, lambda d: layer_norm(d)),
    (W, lambda d: layer_norm(X, d)),
    (W, lambda d: layer_norm(X, None, d)),
    (X, lambda d: layer_norm_forward(d)),
    (X, lambda d: layer_norm_backward(d, X, None, S, S)),
    (X, lambda d: layer_norm_backward(X, d, None, S, S)),
    (W, lambda d: layer_norm_backward(X, X, d, S, S)),
    (S, lambda d: layer_norm_backward(X, X, None, d, S)),
    (S, lambda d: layer_norm_backward(X, X, None, S, d)),
    (Z, lambda d: balance_loss(d, E)),
    (Z, lambda d: balance_forward(d, E)),
    (Z, lambda d: balance_fused(d, E)),
    (G, lambda d: balance_fused(Z, E, grad_output=d)),
    (Z, lambda d: balance_backward(d, C, N, 2)),
    (G, lambda d: balance_backward(Z, C, N, 2, grad_output=d)),
    (L, lambda d: beam_select(d, B)),
    (B, lambda d: beam_select(L, d)),
    (T, lambda d: beam_reorder([T, d], P)),
    (T, lambda d: beam_reorder([T], P, out=[d])),
]


@pytest.mark.parametrize("t,call", CALLS)
def test_forward_mode_tangents_are_refused(t, call):
    with fw.dual_level():
        with pytest.raises(NotImplementedError, match="forward-mode"):
            call(fw.make_dual(t.clone(), torch.ones_like(t)))
        with pytest.raises(ValueError, match="CUDA"):  # without a tangent it is only the device that is wrong
            call(t.clone())


@pytest.mark.parametrize("inputs,call", [
    ((X,), lambda x: layer_norm_forward(x, stats=False)["y"]),
    ((X,), lambda x: layer_norm_backward(x, x, None, S, S)["grad_x"]),
    ((Z, E), lambda z, e: balance_forward(z, e)["loss"]),
    ((Z, E), lambda z, e: balance_fused(z, e)["loss"]),
    ((Z,), lambda z: balance_backward(z, C, N, 2)["grad_logits"]),
    ((L, B), lambda z, s: beam_select(z, s)["tokens"]),
    ((T, P), lambda t, p: beam_reorder([t], p)[0]),
])
def test_traces_of_the_calls_on_their_own_are_refused(inputs, call):
    with pytest.raises(RuntimeError, match="cannot be traced"):
        torch.jit.trace(call, tuple(t.clone() for t in inputs), check_trace=False)
