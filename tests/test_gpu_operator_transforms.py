"""Torch's transforms and the operators beside the head, on the GPU."""
import pytest
import torch
import torch.autograd.forward_ad as fw

from tests.op_util import normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_tangents_are_refused(grad):
    """Through the autograd functions too."""
    from lm_head_linear_chunked_gb300.balance_loss import balance_loss
    from lm_head_linear_chunked_gb300.layer_norm import LayerNorm, layer_norm
    x, z = normal((5, 64), 1), normal((1, 30, 8), 2)
    experts = z.topk(2, dim=-1).indices
    module = LayerNorm(64, device="cuda")
    with fw.dual_level():
        def dual(t):
            return fw.make_dual(t.clone().requires_grad_(grad), torch.ones_like(t))
        for call in (lambda: layer_norm(dual(x)), lambda: layer_norm(x, dual(x[0])), lambda: layer_norm(x, None, dual(x[0])),
                     lambda: module(dual(x)), lambda: balance_loss(dual(z), experts)):
            with pytest.raises(NotImplementedError):
                call()
        assert torch.equal(layer_norm(x), layer_norm(x.clone().requires_grad_(True)))  # those without go on


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.filterwarnings("ignore::torch.jit.TracerWarning", "ignore::DeprecationWarning")
def test_a_trace_computes_with_its_own_inputs(grad):
    """The recorded calls run on what the trace is given later, gradients included."""
    from lm_head_linear_chunked_gb300.balance_loss import balance_loss
    from lm_head_linear_chunked_gb300.layer_norm import layer_norm
    w = normal(64, 3).requires_grad_(grad)
    x, z = (normal(s, 4).requires_grad_(grad) for s in ((5, 64), (1, 30, 8)))
    experts = z.detach().topk(2, dim=-1).indices

    def both(x, z, w):
        return layer_norm(x, w) + 0, balance_loss(z, experts)[0] + 0

    traced = torch.jit.trace(both, (x, z, w), check_trace=False)
    for seed in (5, 6):
        x, z = (normal(s, seed).requires_grad_(grad) for s in ((5, 64), (1, 30, 8)))
        got, want = traced(x, z, w), both(x, z, w)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        if grad:
            a, b = (torch.autograd.grad(r[0].sum() + r[1], (x, z, w)) for r in (got, want))
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.filterwarnings("ignore::torch.jit.TracerWarning", "ignore::DeprecationWarning")
def test_gradients_inside_a_trace_are_refused():
    """The trace has no node for an autograd function's backward."""
    from lm_head_linear_chunked_gb300.balance_loss import balance_loss
    from lm_head_linear_chunked_gb300.layer_norm import layer_norm
    x, z = (normal(s, 7).requires_grad_(True) for s in ((5, 64), (1, 30, 8)))
    experts = z.detach().topk(2, dim=-1).indices
    for f, t in ((lambda x: torch.autograd.grad(layer_norm(x).sum(), x)[0], x),
                 (lambda z: torch.autograd.grad(balance_loss(z, experts)[0], z)[0], z)):
        with pytest.raises(RuntimeError, match="cannot be traced"):
            torch.jit.trace(f, (t,), check_trace=False)
