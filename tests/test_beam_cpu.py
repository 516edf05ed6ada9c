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


def test_outputs_that_share_memory_are_refused():
    """Two blocks would write the same element: an output with itself, and two outputs, their ranges interleaved or not."""
    room = torch.zeros(20, 4, 5)
    wide = torch.zeros(6, 3, 4, 5)
    one = torch.zeros(4, 5)
    for outs in ([one.expand(6, 4, 5)], [torch.zeros(6, 1, 5).expand(6, 4, 5)],
                 [torch.zeros(100).as_strided((6, 4, 5), (10, 5, 1))], [torch.zeros(100).as_strided((6, 4, 5), (8, 2, 2))],
                 [room[:6], room[:6]], [room[:6], room[5:11]], [room[6:12], room[:6], room[11:17]],
                 [wide[:, 0], wide[:, 0]], [wide[:, 0], wide[:, 1], wide[:, 1]],
                 [wide[:, 0], wide.flatten(1)[:, 19:39].unflatten(1, (4, 5))],
                 [wide[:, 0], wide[:, 0].transpose(1, 2).contiguous().transpose(1, 2), wide[:, 0]]):
        with pytest.raises(ValueError, match="overlap"):
            beam_reorder([X] * len(outs), P, out=outs)


def test_outputs_beside_each_other_go_on():
    """Views of one buffer that share no element: only the device is wrong."""
    wide = torch.zeros(6, 3, 4, 5)
    last = torch.zeros(6, 4, 5, 2)
    inner = torch.zeros(6, 4, 3, 5)
    part = torch.zeros(6, 4, 9, 5)
    for outs in ([wide[:, 0], wide[:, 1], wide[:, 2]], [last[..., 0], last[..., 1]], [inner[:, :, 0], inner[:, :, 2]],
                 [wide.flatten(1)[:, 1:21].unflatten(1, (4, 5)), wide.flatten(1)[:, 21:41].unflatten(1, (4, 5))],
                 [part[:, :, 0], part[:, :, 1]], [torch.zeros(12, 4, 5)[::2], torch.zeros(6, 4, 5)]):
        with pytest.raises(ValueError, match="CUDA"):
            beam_reorder([X] * len(outs), P, out=outs)
    # of another width, and of one element a row
    both = torch.zeros(6, 21)
    with pytest.raises(ValueError, match="CUDA"):
        beam_reorder([X, X[:, 0, 0]], P, out=[both[:, 1:].unflatten(1, (4, 5)), both[:, 0]])
    with pytest.raises(ValueError, match="overlap"):
        beam_reorder([X, X[:, 0, 0]], P, out=[both[:, 1:].unflatten(1, (4, 5)), both[:, 20]])


def test_overlap_against_all_addresses():
    """Random strided outputs in one buffer: refused exactly where two elements share an address (where the strides
    of an output nest, as those of views do; others are refused)."""
    import itertools
    import random
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(400):
        buf = torch.zeros(2000)
        rows, outs, cells, nested = 2, [], [], True
        for _ in range(rng.randint(1, 3)):
            shape = (rows, *(rng.randint(1, 3) for _ in range(rng.randint(0, 2))))
            steps = [rng.choice((1, 2, 3, 4, 6, 12, 24, 40)) for _ in shape]
            if rng.random() < 0.5:
                steps.sort(reverse=True)
            start = rng.randint(0, 60)
            outs.append(buf.as_strided(shape, steps, start))
            cells += [start + sum(i * s for i, s in zip(at, steps)) for at in itertools.product(*map(range, shape))]
            reach = 1
            for s, n in sorted((s, n) for s, n in zip(steps, shape) if n > 1):
                nested &= s >= reach
                reach += (n - 1) * s
        shared = len(set(cells)) < len(cells)
        with pytest.raises(ValueError) as e:
            beam_reorder([torch.zeros(2, *o.shape[1:]) for o in outs], torch.zeros(1, 2, dtype=torch.int64), out=outs)
        refused = "overlap" in str(e.value)
        assert refused == (shared or not nested), ([(o.shape, o.stride(), o.storage_offset()) for o in outs])
        seen[refused] += 1
    assert min(seen.values()) > 50


def test_outputs_between_the_states_go_on():
    """One buffer that holds both sets, in any dimension: no element of an output is one of a state's."""
    for d in range(1, 5):
        both = torch.zeros(6, 4, 3, 5).unsqueeze(d).expand(*(2 if i == d else -1 for i in range(5))).contiguous()
        a, b = both.unbind(d)
        for s, o in ((a, b), (b, a)):
            with pytest.raises(ValueError, match="CUDA"):
                beam_reorder([s], P, out=[o])
        for s, o in ((a, a), (b, b)):
            with pytest.raises(ValueError, match="overlaps the states"):
                beam_reorder([s], P, out=[o])
    both = torch.zeros(6, 2, 9, 5)
    with pytest.raises(ValueError, match="CUDA"):
        beam_reorder([both[:, 0, :1].expand(6, 4, 5)], P, out=[both[:, 1, :4]])  # a state of one row, read four times
    with pytest.raises(ValueError, match="overlaps the states"):
        beam_reorder([both[:, 0, :1].expand(6, 4, 5)], P, out=[both[:, 0, :4]])


def test_states_and_outputs_against_all_addresses():
    """Random strided states and outputs in one buffer: refused where an element of an output is one of a state's
    (or, for a state whose strides do not nest, where their ranges meet)."""
    import itertools
    import random
    rng = random.Random(6)
    seen = {True: 0, False: 0}
    while min(seen.values()) < 150:
        buf = torch.zeros(3000)
        inner = tuple(rng.randint(1, 3) for _ in range(rng.randint(0, 2)))
        sides, cells, nested, ranges = [], [], [], []
        for side in range(2):
            shape = (2, *inner)
            steps = [rng.choice((0, 1, 2, 3, 4, 6, 12, 24, 40)[side:]) for _ in shape]
            if side or rng.random() < 0.5:
                steps.sort(reverse=True)
            start = rng.randint(0, 60)
            sides.append(buf.as_strided(shape, steps, start))
            cells.append({start + sum(i * s for i, s in zip(at, steps)) for at in itertools.product(*map(range, shape))})
            reach, ok = 1, True
            for s, n in sorted((s, n) for s, n in zip(steps, shape) if n > 1 and s):
                ok &= s >= reach
                reach += (n - 1) * s
            nested.append(ok)
            ranges.append((min(cells[-1]), max(cells[-1])))
        if not nested[1] or any(n > 1 and s == 0 for s, n in zip(sides[1].stride(), sides[1].shape)):
            continue
        with pytest.raises(ValueError) as e:
            beam_reorder([sides[0]], torch.zeros(1, 2, dtype=torch.int64), out=[sides[1]])
        refused = "overlaps the states" in str(e.value)
        meet = ranges[0][0] <= ranges[1][1] and ranges[1][0] <= ranges[0][1]
        assert refused == bool(cells[0] & cells[1] if nested[0] else meet), [(o.shape, o.stride(), o.storage_offset()) for o in sides]
        seen[refused] += 1


def test_conjugate_and_negative_views_as_outputs_are_refused():
    z = torch.zeros(6, 4, dtype=torch.complex64)
    for state, out in ((z, z.clone().conj()), (z.real, z.clone().conj().imag)):
        with pytest.raises(ValueError, match="view"):
            beam_reorder([state], P, out=[out])
