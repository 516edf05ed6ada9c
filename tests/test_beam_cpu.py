"""Refusals of beam selection and reordering, without a GPU."""
import pytest
import torch

import __graft_entry__
import lm_head_linear_chunked_gb300 as lce
from lm_head_linear_chunked_gb300._native import native
from lm_head_linear_chunked_gb300.beam import beam_reorder, beam_select

A = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


SELECT = dict(items=2, beams=3, V=100, n_out=6, dtype=lce.BF16, logits=A, ld=100, scores=A, finished=None, pad_token=0,
              eos_token=-1, out_scores=A, out_tokens=A, out_parents=A, out_finished=None, ws=A, ws_bytes=1 << 24,
              stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(items=0), 1), (dict(beams=0), 1), (dict(V=0), 1), (dict(n_out=0), 1), (dict(beams=65), 2), (dict(n_out=65), 2),
    (dict(items=30000), 2), (dict(items=2**62), 2), (dict(V=2**31, ld=2**31), 2), (dict(V=1, n_out=4), 2),
    (dict(dtype=3), 1), (dict(logits=None), 1), (dict(logits=A + 1), 1), (dict(ld=99), 1), (dict(scores=None), 1),
    (dict(scores=A + 2), 1), (dict(out_scores=None), 1), (dict(out_tokens=A + 4), 1), (dict(out_parents=None), 1),
    (dict(ws=None), 1), (dict(ws=A + 8), 1), (dict(ws_bytes=1000), 3),
])
def test_select_refusals(kw, code):
    with pytest.raises(lce.LCEError) as e:
        lce.lce_beam_select(*{**SELECT, **kw}.values())
    assert e.value.status == code


def state(**kw):
    s = lce.BeamState(A, 2 * A, 64, 64, 1, 0, 0, 1, 0, 0, 64)
    for k, v in kw.items():
        setattr(s, k, v)
    return (lce.BeamState * 1)(s)


@pytest.mark.parametrize("kw,code", [
    (dict(items=0), 1), (dict(beams=0), 1), (dict(out_beams=-1), 1), (dict(parents=None), 1), (dict(parents=A + 4), 1),
    (dict(n_states=-1), 1), (dict(states=None), 1), (dict(status=A + 2), 1), (dict(items=2**31), 2),
    (dict(states=state(src=None)), 1), (dict(states=state(dst=None)), 1), (dict(states=state(n1=-1)), 1),
    (dict(states=state(run_bytes=-8)), 1), (dict(states=state(n1=2**20, run_bytes=2**12)), 2),
])
def test_reorder_refusals(kw, code):
    args = dict(items=2, beams=3, out_beams=3, parents=A, states=state(), n_states=1, status=None, stream=None)
    args.update(kw)
    with pytest.raises(lce.LCEError) as e:
        lce.lce_beam_reorder(*args.values())
    assert e.value.status == code


def test_nothing_to_move_enqueues_nothing():
    lce.lce_beam_reorder(2, 3, 3, A, state(run_bytes=0, src=None, dst=None), 1, None, None)
    lce.lce_beam_reorder(2, 3, 3, A, None, 0, None, None)
    assert beam_reorder([], torch.zeros((1, 2), dtype=torch.int64)) == []


def test_workspace_size():
    assert lce.lce_beam_workspace_size(1, 4, 151936, 8) < 1 << 20
    assert lce.lce_beam_workspace_size(64, 64, 151936, 64) < 1 << 24
    with pytest.raises(lce.LCEError):
        lce.lce_beam_workspace_size(1, 1, 3, 4)


Z = torch.zeros(2, 3, 20)
S = torch.zeros(2, 3)
P = torch.zeros(2, 3, dtype=torch.int64)
X = torch.zeros(6, 4, 5)


@pytest.mark.parametrize("call,error", [
    (lambda: beam_select(Z, S), ValueError),                                  # not on a GPU
    (lambda: beam_select(Z.double(), S), TypeError),
    (lambda: beam_select(Z[0], S), ValueError),
    (lambda: beam_select(Z[:, :, :0], S), ValueError),
    (lambda: beam_select(Z, S[:1]), ValueError),
    (lambda: beam_select(Z, S.half()), TypeError),
    (lambda: beam_select(Z, S, finished=S), TypeError),
    (lambda: beam_select(Z, S, finished=S[:1] > 0), ValueError),
    (lambda: beam_select(Z, S, n=0), ValueError),
    (lambda: beam_select(Z, S, eos_token=-1), ValueError),
    (lambda: beam_reorder([X], P), ValueError),                               # not on a GPU
    (lambda: beam_reorder([X], P.int()), ValueError),
    (lambda: beam_reorder([X], P[0]), ValueError),
    (lambda: beam_reorder([X[:5]], P), ValueError),
    (lambda: beam_reorder([X, X[:4]], P), ValueError),
    (lambda: beam_reorder([X], P, out=[]), ValueError),
    (lambda: beam_reorder([X], P, out=[X[:, :3]]), ValueError),
    (lambda: beam_reorder([X], P, out=[X.double()]), TypeError),
])
def test_front_end_refusals(call, error):
    with pytest.raises(error):
        call()


def test_overlap_is_refused():
    both = torch.zeros(10, 4, 5)
    for a, b in ((both[:6], both[:6]), (both[:6], both[4:]), (both[4:], both[:6])):
        with pytest.raises(ValueError, match="overlaps"):
            beam_reorder([a], P, out=[b])


def test_ranges():
    overlap = native().overlap
    assert not overlap([]) and not overlap([(0, 8, 0), (8, 16, 1), (16, 24, 0)])
    assert not overlap([(0, 8, 0), (4, 12, 0), (12, 20, 1)])
    assert overlap([(0, 100, 0), (4, 12, 0), (50, 60, 1)]) and overlap([(5, 6, 1), (5, 6, 0)])


def test_layout_of_a_row():
    """(outer runs, strides, inner runs, strides, run) in bytes, of 4-byte elements."""
    x = torch.zeros(6, 8, 40, 16)
    y = torch.zeros(6, 8, 64, 16)
    layout = native().layout
    assert layout(x, torch.zeros(6, 8, 40, 16)) == (1, 0, 0, 1, 0, 0, 4 * 8 * 40 * 16)
    assert layout(x[:, :, :7], y[:, :, :7]) == (1, 0, 0, 8, 4 * 640, 4 * 1024, 4 * 7 * 16)
    assert layout(x[:, :, :1, :1], y[:, :, :1, :1]) == (1, 0, 0, 8, 4 * 640, 4 * 1024, 4)
    assert layout(x[:, :, :, ::2], y[:, :, :40, ::2]) == (8, 4 * 640, 4 * 1024, 320, 8, 8, 4)
    assert layout(x[:, ::2, ::2, ::3], x[:, ::2, ::2, ::3]) is None
    assert layout(x[:, 0].bfloat16(), y[:, 0, :40].bfloat16()) == (1, 0, 0, 1, 0, 0, 2 * 40 * 16)
