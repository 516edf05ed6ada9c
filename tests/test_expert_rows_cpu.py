"""Rows sorted by expert, without a GPU: the C ABI's host checks and the
Python front end's."""
import pytest
import torch

import __graft_entry__
import lm_head_linear_chunked_gb300 as lce
from lm_head_linear_chunked_gb300.expert_rows import combine, combine_backward, dispatch, dispatch_backward, expert_plan

A = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def plan(**kw):
    args = dict(T=4, k=2, E=8, align=1, experts=A, index_bytes=8, mask=None, positions=A, slots=A, counts=A, offsets=A, ws=A,
                ws_bytes=1 << 20, stream=None)
    args.update(kw)
    lce.lce_expert_plan(*args.values())


def spread(**kw):
    args = dict(T=4, k=2, H=64, R=8, dtype=lce.BF16, x=A, ldx=64, positions=A, slots=A, rows=A, ldr=64, stream=None)
    args.update(kw)
    lce.lce_expert_dispatch(*args.values())


def spread_bwd(**kw):
    args = dict(T=4, k=2, H=64, R=8, dtype=lce.BF16, grad_rows=A, ldr=64, positions=A, grad_x=A, ldx=64, stream=None)
    args.update(kw)
    lce.lce_expert_dispatch_backward(*args.values())


def join(**kw):
    args = dict(T=4, k=2, H=64, R=8, dtype=lce.BF16, wtype=lce.F32, rows=A, ldr=64, weights=A, positions=A, y=A, ldy=64, stream=None)
    args.update(kw)
    lce.lce_expert_combine(*args.values())


def join_bwd(**kw):
    args = dict(T=4, k=2, H=64, R=8, dtype=lce.BF16, wtype=lce.F32, grad_y=A, ldg=64, rows=A, ldr=64, weights=A, positions=A,
                slots=A, grad_rows=A, ldgr=64, grad_weights=A, stream=None)
    args.update(kw)
    lce.lce_expert_combine_backward(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(k=0), 1), (dict(E=0), 1), (dict(align=0), 1), (dict(k=9), 2), (dict(E=1025), 2), (dict(align=1025), 2),
    (dict(T=2**30, k=8), 2), (dict(index_bytes=1), 1), (dict(experts=None), 1), (dict(experts=A + 4), 1), (dict(positions=None), 1),
    (dict(positions=A + 2), 1), (dict(slots=None), 1), (dict(slots=A + 1), 1), (dict(counts=None), 1), (dict(counts=A + 4), 1),
    (dict(offsets=None), 1), (dict(offsets=A + 4), 1), (dict(ws=None), 1), (dict(ws=A + 8), 1), (dict(ws_bytes=100), 3)])
def test_plan_refusals(kw, code):
    with pytest.raises(lce.LCEError) as e:
        plan(**kw)
    assert e.value.status == code


SIZES = [(dict(T=-1), 1), (dict(k=0), 1), (dict(H=0), 1), (dict(R=-1), 1), (dict(dtype=4), 1), (dict(k=1025), 2),
         (dict(H=(1 << 20) + 1), 2), (dict(T=2**31), 2), (dict(R=2**31), 2), (dict(T=2**30, k=2), 2), (dict(positions=None), 1),
         (dict(positions=A + 2), 1)]


@pytest.mark.parametrize("call,kw,code", [
    *[(f, kw, code) for f in (spread, spread_bwd, join, join_bwd) for kw, code in SIZES],
    *[(spread, kw, 1) for kw in (dict(x=None), dict(x=A + 1), dict(ldx=63), dict(rows=None), dict(rows=A + 1), dict(ldr=63),
                                 dict(slots=None), dict(slots=A + 2))],
    *[(spread_bwd, kw, 1) for kw in (dict(grad_rows=None), dict(grad_rows=A + 1), dict(ldr=63), dict(grad_x=None), dict(ldx=0))],
    *[(join, kw, 1) for kw in (dict(rows=None), dict(ldr=63), dict(weights=A + 2), dict(y=None), dict(y=A + 1), dict(ldy=63),
                               dict(wtype=9))],
    (join, dict(wtype=lce.F16), 2), (join_bwd, dict(wtype=lce.F16), 2),
    *[(join_bwd, kw, 1) for kw in (dict(grad_y=None), dict(ldg=63), dict(rows=None), dict(ldr=63), dict(weights=A + 2), dict(slots=None),
                                   dict(grad_rows=A + 1), dict(ldgr=63), dict(grad_weights=A + 2))],
])
def test_move_refusals(call, kw, code):
    with pytest.raises(lce.LCEError) as e:
        call(**kw)
    assert e.value.status == code


def test_nothing_to_do_enqueues_nothing():
    join(T=0, positions=None, y=None)
    spread_bwd(T=0, positions=None, grad_x=None)
    spread(T=0, R=0, positions=None, x=None, slots=None, rows=None)
    join_bwd(grad_rows=None, grad_weights=None)


def test_rows_of_a_plan():
    assert lce.lce_expert_rows(10, 2, 4, 1) == 20
    assert lce.lce_expert_rows(0, 2, 4, 1) == 0
    assert lce.lce_expert_rows(10, 2, 4, 16) == 80  # 20 + 4 * 15
    for args in ((-1, 2, 4, 1), (1, 0, 4, 1), (1, 5, 4, 1), (1, 2, 4, 0)):
        with pytest.raises(lce.LCEError):
            lce.lce_expert_rows(*args)
    assert lce.lce_expert_plan_workspace_size(1 << 20, 8, 1024) < 1 << 21  # bounded whatever the tokens


E = torch.zeros(4, 2, dtype=torch.int64)
X = torch.zeros(4, 16, dtype=torch.bfloat16)
R = torch.zeros(8, 16, dtype=torch.bfloat16)
W = torch.zeros(4, 2)
P = {"positions": torch.zeros(4, 2, dtype=torch.int32), "slots": torch.zeros(8, dtype=torch.int32)}


def other(**kw):
    return {**P, **kw}


@pytest.mark.parametrize("call,error", [
    (lambda: expert_plan(E, 8), ValueError),                                    # not on a GPU
    (lambda: expert_plan(E.float(), 8), TypeError),
    (lambda: expert_plan(E[:, :0], 8), ValueError),
    (lambda: expert_plan(E, 8, torch.ones(3, dtype=torch.bool)), ValueError),
    (lambda: expert_plan(E, 8, torch.ones(4)), TypeError),
    (lambda: expert_plan(E, 0), lce.LCEError),
    (lambda: expert_plan(E, 1), lce.LCEError),                                  # more slots than experts
    (lambda: expert_plan(E, 8, align=0), lce.LCEError),
    (lambda: dispatch(X, P), ValueError),                                       # not on a GPU
    (lambda: dispatch(X[:3], P), ValueError),
    (lambda: dispatch(X.double(), P), TypeError),
    (lambda: dispatch(X[:, :0], P), ValueError),
    (lambda: dispatch(X, other(positions=P["positions"].long())), TypeError),
    (lambda: dispatch(X, other(positions=P["positions"].t())), ValueError),
    (lambda: dispatch(X, other(slots=P["slots"][::2])), ValueError),
    (lambda: dispatch(X, other(slots=P["slots"].long())), TypeError),
    (lambda: dispatch_backward(R[:7], P), ValueError),
    (lambda: dispatch_backward(R, P), ValueError),                              # not on a GPU
    (lambda: combine(R, W, P), ValueError),                                     # not on a GPU
    (lambda: combine(R[:5], W, P), ValueError),
    (lambda: combine(R[0], W, P), ValueError),
    (lambda: combine(R, W[:, :1], P), ValueError),
    (lambda: combine(R, W.half(), P), TypeError),
    (lambda: combine(R.double(), W, P), TypeError),
    (lambda: combine_backward(X, R, W, P), ValueError),                         # not on a GPU
    (lambda: combine_backward(X[:2], R, W, P), ValueError),
    (lambda: combine_backward(X.float(), R, W, P), TypeError),
    (lambda: combine_backward(X[:, :8], R, W, P), ValueError),
    (lambda: combine_backward(X, R[:7], W, P), ValueError),
])
def test_front_end_refusals(call, error):
    with pytest.raises(error):
        call()
