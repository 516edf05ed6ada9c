"""Embedding without a GPU: the C ABI's host checks, the Python front end's
checks, and the formula of the gradient against differences."""
import pytest
import torch

import __graft_entry__
import lm_head_linear_chunked_gb300 as lce
from lm_head_linear_chunked_gb300.embedding import Embedding, embedding, embedding_backward
from tests.row_refs import embedding_grad_ref

A = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def fwd(**kw):
    args = dict(N=4, V=10, H=64, dtype=lce.BF16, tokens=A, index_bytes=8, weight=A, ldw=64, scale=1.0,
                padding_token=lce.NO_PADDING, y=A, ldy=64, status=None, stream=None)
    args.update(kw)
    lce.lce_embedding_forward(*args.values())


def bwd(**kw):
    args = dict(N=4, V=10, H=64, dtype=lce.BF16, gtype=lce.BF16, tokens=A, index_bytes=8, grad_y=A, ldg=64, scale=1.0,
                padding_token=lce.NO_PADDING, grad_weight=A, ldgw=64, ws=A, ws_bytes=1 << 20, stream=None, flags=0)
    args.update(kw)
    lce.lce_embedding_backward(*args.values())


SIZES = [(dict(N=-1), 1), (dict(V=0), 1), (dict(H=0), 1), (dict(dtype=5), 1), (dict(N=2**31), 2), (dict(V=2**31 - 1), 2),
         (dict(H=(1 << 20) + 1), 2), (dict(tokens=None), 1), (dict(tokens=A + 4), 1), (dict(index_bytes=2), 1)]


@pytest.mark.parametrize("kw,code", SIZES + [(dict(weight=None), 1), (dict(weight=A + 1), 1), (dict(y=None), 1), (dict(ldw=63), 1),
                                             (dict(y=A + 1), 1), (dict(ldy=1), 1), (dict(status=A + 2), 1)])
def test_forward_refusals(kw, code):
    with pytest.raises(lce.LCEError) as e:
        fwd(**kw)
    assert e.value.status == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(grad_y=None), 1), (dict(grad_y=A + 1), 1), (dict(ldg=63), 1), (dict(ldgw=63), 1), (dict(grad_weight=None), 1),
    (dict(grad_weight=A + 1), 1), (dict(ws=None), 1), (dict(ws=A + 8), 1), (dict(ws_bytes=64), 3), (dict(gtype=lce.F16), 2),
    (dict(gtype=7), 1), (dict(flags=lce.ACCUMULATE), 2), (dict(flags=lce.REDUCTION_SUM), 1)])
def test_backward_refusals(kw, code):
    with pytest.raises(lce.LCEError) as e:
        bwd(**kw)
    assert e.value.status == code


def test_no_tokens_enqueue_nothing_in_the_forward():
    fwd(N=0, tokens=None, weight=None, y=None)


def test_workspace_size():
    size = lce.lce_embedding_workspace_size
    N, H = 1 << 20, 4096
    assert size(0, 10, 64) >= 1024
    # two float32 rows of pieces for 32 tokens, a few words for each token, a byte for each vocabulary row
    assert N * H // 4 <= size(N, 151936, H) < N * H // 4 + N * 32 + (1 << 20)
    for args in ((-1, 10, 64), (4, 0, 64), (4, 10, 0)):
        with pytest.raises(lce.LCEError):
            size(*args)


W = torch.zeros(10, 16, dtype=torch.bfloat16)
T = torch.zeros(4, dtype=torch.int64)
D = torch.zeros(4, 16, dtype=torch.bfloat16)
ONE = torch.zeros(20, 16)


@pytest.mark.parametrize("call,error", [
    (lambda: embedding(T, W), ValueError),                       # not on a GPU
    (lambda: embedding(T, W.double()), TypeError),
    (lambda: embedding(T.float(), W), TypeError),
    (lambda: embedding(T.to(torch.int16), W), TypeError),
    (lambda: embedding(T, W[0]), ValueError),
    (lambda: embedding(T, W[:, :0]), ValueError),
    (lambda: embedding_backward(D, T, 10), ValueError),          # not on a GPU
    (lambda: embedding_backward(D[:3], T, 10), ValueError),
    (lambda: embedding_backward(D[:, :0], T, 10), ValueError),
    (lambda: embedding_backward(D, T, 0), ValueError),
    (lambda: embedding_backward(D.double(), T, 10), TypeError),
    (lambda: embedding_backward(D, T, 10, dtype=torch.float16), TypeError),
    (lambda: embedding_backward(D, T, 10, accumulate=True), ValueError),
    (lambda: embedding_backward(D, T, 10, out=W, accumulate=True), TypeError),
    (lambda: embedding_backward(D, T, 10, out=W[:9]), ValueError),
    (lambda: embedding_backward(D, T, 10, dtype=torch.float32, out=W), TypeError),
    (lambda: embedding_backward(D, T, 10, out=W[:1].expand(10, 16)), ValueError),
    (lambda: embedding_backward(D, T, 10, out=torch.zeros(16, 10, dtype=torch.bfloat16).t()), ValueError),
    (lambda: embedding_backward(ONE[1:9], T.repeat(2), 10, out=ONE[8:18]), ValueError),   # overlap
    (lambda: Embedding(0, 4), ValueError),
    (lambda: Embedding(4, 0), ValueError),
])
def test_front_end_refusals(call, error):
    with pytest.raises(error):
        call()


def test_an_output_that_overlaps_the_gradient():
    for a, b, overlap in ((0, 4, False), (1, 4, True), (4, 4, True), (13, 4, True), (14, 4, False), (5, 0, False)):
        with pytest.raises(ValueError, match="overlap" if overlap else "CUDA"):
            embedding_backward(ONE[a:a + b], T[:b], 10, out=ONE[4:14])


SIDE = torch.zeros(20, 40)
BITS = SIDE.view(torch.bfloat16)


@pytest.mark.parametrize("dy,out,overlap", [
    (SIDE[2:6, 16:32], SIDE[:10, :16], False),             # other columns of one buffer
    (SIDE[2:6, 24:40], SIDE[5:15, 8:24], False),
    (SIDE[6:10, :16], SIDE[:10, 16:32], False),
    (SIDE[6:10, :16], SIDE[:10, 15:31], True),
    (SIDE[2:6, 15:31], SIDE[:10, :16], True),
    (SIDE[::2][:4, 24:40], SIDE[:10, 8:24], False),        # every other row
    (SIDE[2:3, 16:32].expand(4, 16), SIDE[:10, :16], False),
    (SIDE.reshape(-1)[30:190].view(4, 40)[:, :16], SIDE[:10, :16], True),    # reaches into the next row's first columns
    (SIDE.reshape(-1)[:288].view(8, 36)[:4, 16:32], SIDE[:10, :16], True),   # rows of another length
    (BITS[2:6, 32:48], SIDE[:10, :16], False),             # 16-bit rows beside float32 ones
    (BITS[2:6, 31:47], SIDE[:10, :16], True),
])
def test_an_output_beside_the_gradient(dy, out, overlap):
    with pytest.raises(ValueError, match="overlap" if overlap else "CUDA"):
        embedding_backward(dy, T, 10, out=out)


def test_module_parameters():
    m = Embedding(6, 4, padding_idx=2, dtype=torch.bfloat16)
    assert m.weight.shape == (6, 4) and m.weight.dtype == torch.bfloat16 and not m.weight[2].any()
    Embedding(6, 4, padding_idx=-1)


def test_the_gradient_formula_against_differences():
    """The lookup is linear, so differences are exact up to 2^-52 / h."""
    g = torch.Generator().manual_seed(1)
    w, dy = torch.randn(5, 3, dtype=torch.float64, generator=g), torch.randn(8, 3, dtype=torch.float64, generator=g)
    t = torch.tensor([0, 3, 3, 1, 4, 3, 0, 2])
    grad = embedding_grad_ref(dy, t, 5, 1.5, padding=2)[0]
    for i in range(15):
        e = torch.zeros(15, dtype=torch.float64)
        e[i] = 1e-3
        loss = [(1.5 * (w + s * e.view(5, 3))[t] * dy)[t != 2].sum() for s in (1, -1)]
        assert abs((loss[0] - loss[1]) / 2e-3 - grad.reshape(-1)[i]) < 1e-10
