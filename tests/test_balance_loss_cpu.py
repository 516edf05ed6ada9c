"""Refusals of the balance loss, without a GPU: the C ABI's host checks and
the Python front end's checks."""
import pytest
import torch

import __graft_entry__
import lm_head_linear_chunked_gb300 as lce
from lm_head_linear_chunked_gb300.balance_loss import balance_backward, balance_forward, balance_fused, balance_loss

A = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


FWD = dict(groups=2, T=10, E=8, k=2, dtype=lce.F32, logits=A, group_stride=80, token_stride=8, experts=A,
           index_bytes=8, mask=None, mask_group_stride=0, loss=A, group_loss=None, counts=A, n_valid=A, ws=A,
           ws_bytes=1 << 24, stream=None, flags=0)
FUSED = dict(groups=2, T=10, E=8, k=2, dtype=lce.F32, logits=A, group_stride=80, token_stride=8, experts=A,
             index_bytes=8, mask=None, mask_group_stride=0, grad_scale=1.0, d_grad_output=None, loss=A,
             group_loss=None, counts=A, n_valid=A, grad_logits=A, ws=A, ws_bytes=1 << 24, stream=None, flags=0)
BWD = dict(groups=2, T=10, E=8, k=2, dtype=lce.F32, logits=A, group_stride=80, token_stride=8, counts=A, n_valid=A,
           mask=None, mask_group_stride=0, grad_scale=1.0, d_grad_output=None, grad_logits=A, stream=None, flags=0)

COMMON = [(dict(groups=0), 1), (dict(T=0), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=9), 2), (dict(groups=65536), 2),
          (dict(E=1025, token_stride=2000), 2), (dict(T=2**31), 2), (dict(dtype=7), 1), (dict(logits=None), 1),
          (dict(logits=A + 2), 1), (dict(token_stride=7), 1), (dict(group_stride=-1), 1),
          (dict(mask_group_stride=-1), 1), (dict(flags=2), 1), (dict(counts=None), 1), (dict(n_valid=None), 1),
          (dict(counts=A + 4), 1)]


@pytest.mark.parametrize("call,base", [(lce.lce_balance_forward, FWD), (lce.lce_balance_fused, FUSED),
                                       (lce.lce_balance_backward, BWD)])
@pytest.mark.parametrize("kw,code", COMMON)
def test_common_refusals(call, base, kw, code):
    with pytest.raises(lce.LCEError) as e:
        call(*{**base, **kw}.values())
    assert e.value.status == code


@pytest.mark.parametrize("call,base", [(lce.lce_balance_forward, FWD), (lce.lce_balance_fused, FUSED)])
@pytest.mark.parametrize("kw,code", [(dict(experts=None), 1), (dict(experts=A + 4), 1), (dict(index_bytes=2), 1),
                                     (dict(loss=None), 1), (dict(ws=None), 1), (dict(ws=A + 128), 1),
                                     (dict(ws_bytes=512), 3)])
def test_loss_refusals(call, base, kw, code):
    with pytest.raises(lce.LCEError) as e:
        call(*{**base, **kw}.values())
    assert e.value.status == code


@pytest.mark.parametrize("call,base", [(lce.lce_balance_backward, BWD), (lce.lce_balance_fused, FUSED)])
@pytest.mark.parametrize("kw,code", [(dict(grad_logits=None), 1), (dict(grad_logits=A + 2), 1),
                                     (dict(d_grad_output=A + 1), 1)])
def test_gradient_refusals(call, base, kw, code):
    with pytest.raises(lce.LCEError) as e:
        call(*{**base, **kw}.values())
    assert e.value.status == code


def test_workspace_size():
    assert lce.lce_balance_workspace_size(1, 1, 8, 2) > 0
    assert lce.lce_balance_workspace_size(1, 1 << 30, 256, 8) < 1 << 24  # bounded whatever the tokens
    with pytest.raises(lce.LCEError):
        lce.lce_balance_workspace_size(1, 10, 8, 9)


Z = torch.zeros(2, 10, 8)
E = torch.zeros(2, 10, 2, dtype=torch.int64)
M = torch.ones(10, dtype=torch.bool)
C = torch.zeros(2, 8, dtype=torch.int64)
N = torch.zeros(2, dtype=torch.int64)


@pytest.mark.parametrize("call,error", [
    (lambda: balance_loss(Z, E), ValueError),                                 # not on a GPU
    (lambda: balance_loss(Z.double(), E), TypeError),
    (lambda: balance_loss(Z[0, 0], E[0, 0]), ValueError),
    (lambda: balance_loss(Z[:, :0], E[:, :0]), ValueError),
    (lambda: balance_loss(Z, E.float()), TypeError),
    (lambda: balance_loss(Z, E[:, :9]), ValueError),
    (lambda: balance_loss(Z, E[0]), ValueError),
    (lambda: balance_loss(Z, E[..., :0]), ValueError),
    (lambda: balance_loss(Z, E, M.long()), TypeError),
    (lambda: balance_loss(Z, E, M[:9]), ValueError),
    (lambda: balance_loss(Z, E, M[None].expand(3, 10)), ValueError),
    (lambda: balance_forward(Z, E, reduction="none"), ValueError),
    (lambda: balance_fused(Z, E, grad_output=torch.zeros(2)), ValueError),
    (lambda: balance_backward(Z, C[:1], N, 2), ValueError),
    (lambda: balance_backward(Z, C, N[:1], 2), ValueError),
    (lambda: balance_backward(Z, C.int(), N, 2), TypeError),
    (lambda: balance_backward(Z, C, N, 2), ValueError),
])
def test_front_end_refusals(call, error):
    with pytest.raises(error):
        call()
