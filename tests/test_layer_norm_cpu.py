"""Refusals of layer norm, without a GPU: the C ABI's host checks and the
Python front end's checks of types, shapes and devices."""
import pytest
import torch

import __graft_entry__
import lm_head_linear_chunked_gb300 as lce
from lm_head_linear_chunked_gb300.layer_norm import LayerNorm, layer_norm, layer_norm_backward, layer_norm_forward

A = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def fwd(**kw):
    args = dict(rows=4, H=64, dtype=lce.BF16, wtype=lce.F32, x=A, ldx=64, weight=A, bias=A, eps=1e-5, y=A, ldy=64,
                mean=A, rstd=A, stream=None)
    args.update(kw)
    lce.lce_layer_norm_forward(*args.values())


def bwd(**kw):
    args = dict(rows=4, H=64, dtype=lce.BF16, wtype=lce.F32, grad_y=A, ldg=64, x=A, ldx=64, weight=A, mean=A, rstd=A,
                grad_x=A, ldgx=64, grad_weight=A, grad_bias=A, ws=A, ws_bytes=1 << 20, stream=None)
    args.update(kw)
    lce.lce_layer_norm_backward(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(H=0), 1), (dict(dtype=3), 1), (dict(wtype=-1), 1), (dict(x=None), 1), (dict(y=None), 1),
    (dict(x=A + 1), 1), (dict(weight=A + 2), 1), (dict(bias=A + 1), 1), (dict(mean=None), 1), (dict(rstd=None), 1),
    (dict(mean=A + 2), 1), (dict(ldx=63), 1), (dict(ldy=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(wtype=lce.F16), 2), (dict(dtype=lce.F32, wtype=lce.BF16), 2), (dict(rows=2**31), 2),
    (dict(H=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21), 2),
])
def test_forward_refusals(kw, code):
    with pytest.raises(lce.LCEError) as e:
        fwd(**kw)
    assert e.value.status == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(H=-4), 1), (dict(grad_y=None), 1), (dict(x=None), 1), (dict(mean=None), 1),
    (dict(rstd=None), 1), (dict(ws=None), 1), (dict(ws=A + 16), 1), (dict(ws_bytes=64), 3), (dict(ldg=1), 1),
    (dict(ldgx=1), 1), (dict(grad_weight=A + 2), 1), (dict(grad_x=A + 1), 1), (dict(wtype=lce.F16), 2),
])
def test_backward_refusals(kw, code):
    with pytest.raises(lce.LCEError) as e:
        bwd(**kw)
    assert e.value.status == code


def test_no_rows_enqueue_nothing():
    fwd(rows=0, x=None, y=None)
    bwd(rows=0, grad_weight=None, grad_bias=None, x=None, grad_y=None)


def test_workspace_size():
    one = lce.lce_layer_norm_workspace_size(1, 64)
    assert one >= 2 * 64 * 4
    assert lce.lce_layer_norm_workspace_size(0, 64) == one
    assert lce.lce_layer_norm_workspace_size(1 << 30, 4096) < 1 << 28  # bounded whatever the rows
    with pytest.raises(lce.LCEError):
        lce.lce_layer_norm_workspace_size(4, 0)


X = torch.zeros(4, 16, dtype=torch.bfloat16)
W = torch.zeros(16, dtype=torch.bfloat16)
S = torch.zeros(4)


@pytest.mark.parametrize("call,error", [
    (lambda: layer_norm(X, W), ValueError),                                     # not on a GPU
    (lambda: layer_norm(X.double(), None), TypeError),
    (lambda: layer_norm(X, W[:8]), ValueError),
    (lambda: layer_norm(X, W.half()), TypeError),
    (lambda: layer_norm(X, W, W.float()), TypeError),                           # two types
    (lambda: layer_norm(X, torch.zeros(32, dtype=torch.bfloat16)[::2]), ValueError),
    (lambda: layer_norm(torch.zeros(()), None), ValueError),
    (lambda: layer_norm(torch.zeros(4, 0), None), ValueError),
    (lambda: layer_norm_forward(X, None, W[:3]), ValueError),
    (lambda: layer_norm_backward(X[:2], X, W, S, S), ValueError),
    (lambda: layer_norm_backward(X.float(), X, W, S, S), TypeError),
    (lambda: layer_norm_backward(X, X, W, S[:3], S), ValueError),
    (lambda: layer_norm_backward(X, X, W, S, S.double()), TypeError),
    (lambda: layer_norm_backward(X, X, None, S, S, grad_dtype=torch.float16), TypeError),
    (lambda: layer_norm_backward(X, X, W, S, S), ValueError),
    (lambda: LayerNorm(0), ValueError),
])
def test_front_end_refusals(call, error):
    with pytest.raises(error):
        call()


def test_module_parameters():
    m = LayerNorm(8, dtype=torch.bfloat16)
    assert m.weight.dtype == torch.bfloat16 and bool((m.weight == 1).all()) and not m.bias.any()
    assert LayerNorm(8, bias=False).bias is None
