"""RMS norm without a GPU: the C ABI's host checks, the Python front end's
checks, and the formula of the gradient against differences."""
import pytest
import torch

import __graft_entry__
import lm_head_linear_chunked_gb300 as lce
from lm_head_linear_chunked_gb300.rms_norm import RMSNorm, rms_norm, rms_norm_backward, rms_norm_forward, rms_norm_fp8
from tests.row_refs import rms_backward_ref, rms_ref

A = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def fwd(**kw):
    args = dict(rows=4, H=64, dtype=lce.BF16, wtype=lce.F32, x=A, ldx=64, residual=A, ldr=64, weight=A, eps=1e-6, sum=A,
                lds=64, y=A, ldy=64, rstd=A, stream=None)
    args.update(kw)
    lce.lce_rms_norm_forward(*args.values())


def fp8(**kw):
    args = dict(rows=4, H=64, dtype=lce.BF16, wtype=lce.F32, x=A, ldx=64, residual=A, ldr=64, weight=A, eps=1e-6, sum=A,
                lds=64, q=A, ldq=64, scales=A, group=128, stream=None)
    args.update(kw)
    lce.lce_rms_norm_fp8(*args.values())


def bwd(**kw):
    args = dict(rows=4, H=64, dtype=lce.BF16, wtype=lce.F32, grad_y=A, ldg=64, x=A, ldx=64, weight=A, rstd=A, grad_sum=A,
                ldgs=64, grad_x=A, ldgx=64, grad_weight=A, ws=A, ws_bytes=1 << 20, stream=None)
    args.update(kw)
    lce.lce_rms_norm_backward(*args.values())


INPUTS = [
    (dict(rows=-1), 1), (dict(H=0), 1), (dict(dtype=3), 1), (dict(wtype=-1), 1), (dict(x=None), 1), (dict(x=A + 1), 1),
    (dict(residual=A + 1), 1), (dict(residual=None), 1), (dict(sum=None), 1), (dict(sum=A + 1), 1), (dict(weight=A + 2), 1),
    (dict(ldx=63), 1), (dict(ldr=63), 1), (dict(lds=1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(wtype=lce.F16), 2), (dict(dtype=lce.F32, wtype=lce.BF16), 2), (dict(rows=2**31), 2),
    (dict(H=(1 << 20) + 1, ldx=1 << 21, ldr=1 << 21, lds=1 << 21), 2),
]


@pytest.mark.parametrize("kw,code", INPUTS + [(dict(y=None), 1), (dict(y=A + 1), 1), (dict(ldy=0), 1), (dict(rstd=A + 2), 1)])
def test_forward_refusals(kw, code):
    with pytest.raises(lce.LCEError) as e:
        fwd(**kw)
    assert e.value.status == code


@pytest.mark.parametrize("kw,code", INPUTS + [
    (dict(q=None), 1), (dict(ldq=63), 1), (dict(scales=None), 1), (dict(scales=A + 2), 1), (dict(group=-1), 1),
    (dict(group=64), 2)])
def test_fp8_refusals(kw, code):
    with pytest.raises(lce.LCEError) as e:
        fp8(**kw)
    assert e.value.status == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(H=-4), 1), (dict(grad_y=None), 1), (dict(x=None), 1), (dict(rstd=None), 1), (dict(ws=None), 1),
    (dict(ws=A + 16), 1), (dict(ws_bytes=64), 3), (dict(ldg=1), 1), (dict(ldgx=1), 1), (dict(ldgs=1), 1),
    (dict(grad_weight=A + 2), 1), (dict(grad_x=A + 1), 1), (dict(grad_sum=A + 1), 1), (dict(wtype=lce.F16), 2),
])
def test_backward_refusals(kw, code):
    with pytest.raises(lce.LCEError) as e:
        bwd(**kw)
    assert e.value.status == code


def test_no_rows_enqueue_nothing():
    fwd(rows=0, x=None, residual=None, sum=None, y=None)
    fp8(rows=0, x=None, residual=None, sum=None, q=None, scales=None)
    bwd(rows=0, grad_weight=None, x=None, grad_y=None, rstd=None)


def test_workspace_size():
    one = lce.lce_rms_norm_workspace_size(1, 64)
    assert one >= 64 * 4
    assert lce.lce_rms_norm_workspace_size(0, 64) == one
    assert lce.lce_rms_norm_workspace_size(1 << 30, 4096) < 1 << 28  # bounded whatever the rows
    with pytest.raises(lce.LCEError):
        lce.lce_rms_norm_workspace_size(4, 0)


X = torch.zeros(4, 16, dtype=torch.bfloat16)
W = torch.zeros(16, dtype=torch.bfloat16)
S = torch.zeros(4)


@pytest.mark.parametrize("call,error", [
    (lambda: rms_norm(X, W), ValueError),                                     # not on a GPU
    (lambda: rms_norm(X, W, X), ValueError),
    (lambda: rms_norm(X.double(), None), TypeError),
    (lambda: rms_norm(X, W[:8]), ValueError),
    (lambda: rms_norm(X, W.half()), TypeError),
    (lambda: rms_norm(X, torch.zeros(32, dtype=torch.bfloat16)[::2]), ValueError),
    (lambda: rms_norm(X, W, X[:2]), ValueError),
    (lambda: rms_norm(X, W, X.float()), TypeError),
    (lambda: rms_norm(torch.zeros(()), None), ValueError),
    (lambda: rms_norm(torch.zeros(4, 0), None), ValueError),
    (lambda: rms_norm_forward(X, W[:3]), ValueError),
    (lambda: rms_norm_fp8(X, W, group=32), ValueError),
    (lambda: rms_norm_fp8(X, W), ValueError),
    (lambda: rms_norm_backward(X[:2], X, W, S), ValueError),
    (lambda: rms_norm_backward(X.float(), X, W, S), TypeError),
    (lambda: rms_norm_backward(X, X, W, S[:3]), ValueError),
    (lambda: rms_norm_backward(X, X, W, S.double()), TypeError),
    (lambda: rms_norm_backward(X, X, W, S, X.float()), TypeError),
    (lambda: rms_norm_backward(X, X, W, S, X[:1]), ValueError),
    (lambda: rms_norm_backward(X, X, W, S), ValueError),
    (lambda: RMSNorm(0), ValueError),
])
def test_front_end_refusals(call, error):
    with pytest.raises(error):
        call()


def test_module_parameters():
    m = RMSNorm(8, dtype=torch.bfloat16)
    assert m.weight.dtype == torch.bfloat16 and bool((m.weight == 1).all()) and len(list(m.parameters())) == 1


def test_the_gradient_formula_against_differences():
    """The reference that the kernels are held to, in float64: central differences with step h are off by h^2 times a
    third derivative of order one and by 2^-52 / h, about 1e-10 both at h = 1e-5."""
    g = torch.Generator().manual_seed(1)
    x, w, dy, ds = (torch.randn(s, dtype=torch.float64, generator=g) for s in ((3, 7), (7,), (3, 7), (3, 7)))
    rstd = (x.square().mean(1) + 0.1).rsqrt()
    dx, dw = rms_backward_ref(dy, x, w, rstd, ds)

    def loss(x, w):
        return (rms_ref(x, w, 0.1)[0] * dy).sum() + (x * ds).sum()

    for t, grad in ((x, dx), (w, dw)):
        for i in range(t.numel()):
            e = torch.zeros_like(t).reshape(-1)
            e[i] = 1e-5
            e = e.reshape(t.shape)
            up, down = (loss(x + e, w), loss(x - e, w)) if t is x else (loss(x, w + e), loss(x, w - e))
            assert abs((up - down) / 2e-5 - grad.reshape(-1)[i]) < 1e-8
