"""Torch's transforms and the operators between token ids and the head, without a GPU: forward-mode tangents are refused
instead of lost, and calls that a trace would not see are not traced."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import __graft_entry__
from lm_head_linear_chunked_gb300.embedding import embedding, embedding_backward
from lm_head_linear_chunked_gb300.expert_rows import combine, combine_backward, dispatch, dispatch_backward, expert_plan
from lm_head_linear_chunked_gb300.rms_norm import rms_norm, rms_norm_backward, rms_norm_forward, rms_norm_fp8


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


X, W, S = torch.zeros(4, 16), torch.ones(16), torch.zeros(4)
T, E = torch.zeros(4, dtype=torch.int64), torch.zeros(10, 16)
P = {"positions": torch.zeros(4, 2, dtype=torch.int32), "slots": torch.zeros(8, dtype=torch.int32)}
R, G = torch.zeros(8, 16), torch.zeros(4, 2)

# each with the tensor that gets the tangent, and the call
CALLS = [
    (X, lambda d: rms_norm(d)),
    (W, lambda d: rms_norm(X, d)),
    (X, lambda d: rms_norm(X, None, d)),
    (X, lambda d: rms_norm_forward(d)),
    (X, lambda d: rms_norm_fp8(d)),
    (X, lambda d: rms_norm_fp8(X, None, d)),
    (X, lambda d: rms_norm_backward(d, X, W, S)),
    (X, lambda d: rms_norm_backward(X, d, W, S)),
    (W, lambda d: rms_norm_backward(X, X, d, S)),
    (S, lambda d: rms_norm_backward(X, X, W, d)),
    (X, lambda d: rms_norm_backward(X, X, W, S, d)),
    (E, lambda d: embedding(T, d)),
    (X, lambda d: embedding_backward(d, T, 10)),
    (E, lambda d: embedding_backward(X, T, 10, out=d)),
    (X, lambda d: dispatch(d, P)),
    (R, lambda d: dispatch_backward(d, P)),
    (R, lambda d: combine(d, G, P)),
    (G, lambda d: combine(R, d, P)),
    (X, lambda d: combine_backward(d, R, G, P)),
    (R, lambda d: combine_backward(X, d, G, P)),
    (G, lambda d: combine_backward(X, R, d, P)),
]


@pytest.mark.parametrize("t,call", CALLS)
def test_forward_mode_tangents_are_refused(t, call):
    with fw.dual_level():
        with pytest.raises(NotImplementedError, match="forward-mode"):
            call(fw.make_dual(t.clone(), torch.ones_like(t)))
        with pytest.raises(ValueError, match="CUDA"):  # without a tangent it is only the device that is wrong
            call(t.clone())


@pytest.mark.parametrize("inputs,call", [
    ((X,), lambda x: rms_norm_forward(x, stats=False)["y"]),
    ((X,), lambda x: rms_norm_fp8(x)["scales"]),
    ((X,), lambda x: rms_norm_backward(x, x, None, S)["grad_x"]),
    ((X,), lambda x: embedding_backward(x, T, 10)),
    ((T,), lambda t: expert_plan(t[:, None], 8)["slots"]),
    ((R,), lambda r: dispatch_backward(r, P)),
    ((X,), lambda x: combine_backward(x, R, G, P)["grad_rows"]),
])
def test_traces_of_the_calls_on_their_own_are_refused(inputs, call):
    with pytest.raises(RuntimeError, match="cannot be traced"):
        torch.jit.trace(call, tuple(t.clone() for t in inputs), check_trace=False)
