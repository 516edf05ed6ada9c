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
