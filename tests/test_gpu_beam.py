"""Beam selection and state reordering (beam.py) on the GPU against float64.

Tolerance of a score: one fp32 rounding of it, and the error of lse.  A term
2^t of the sum, t = (z - max) log2 e, is off by at most (2 |t| + 2) 2^-24;
terms with |t| > 40 weigh less than V 2^-40 together, so with sums of 32 in
sequence the logarithm is off by at most E = 128 * 2^-24.  Tokens and parents
have to be those of the float64 order, (score down, beam up, logit down,
token up), except among candidates of different beams whose scores are within
2 E of each other."""
import numpy as np
import pytest
import torch

import lm_head_linear_chunked_gb300 as lce
from tests.op_util import DTYPES, U32, normal

pytestmark = pytest.mark.gpu
E_LSE = 128 * U32


def reference(logits, scores, n, finished, pad):
    """(scores, parents, tokens) of each item's candidates in the definition's order."""
    B, K, V = logits.shape
    z = logits.double().cpu().numpy()
    z = np.where(np.isnan(z), -np.inf, np.minimum(z, float(np.finfo(np.float32).max)))
    s = scores.double().cpu().numpy()
    s = np.where(np.isnan(s), -np.inf, s)
    out = []
    for b in range(B):
        sc, be, to = [], [], []
        for k in range(K):
            if finished is not None and bool(finished[b, k]):
                m = min(V, n)
                sc.append(np.where(np.arange(m) == 0, s[b, k], -np.inf))
                to.append(np.full(m, pad))
            else:
                m = min(V, n + 1)
                x = z[b, k]
                top = x.max()
                at = np.lexsort((np.arange(V), -x))[:m]
                with np.errstate(all="ignore"):
                    log_sum = np.log(np.exp(x - top).sum()) if top > -np.inf else 0.0
                    sc.append(np.where(x[at] > -np.inf, s[b, k] + (x[at] - top) - log_sum, -np.inf))
                to.append(at)
            be.append(np.full(m, k))
        sc, be, to = (np.concatenate(q) for q in (sc, be, to))
        order = np.lexsort((np.arange(len(sc)), be, -sc))  # within a beam already by logit and token
        out.append((sc[order], be[order], to[order]))
    return out


def check(logits, scores, n=None, finished=None, pad=0, eos=None, exact=False):
    from lm_head_linear_chunked_gb300.beam import beam_select
    got = beam_select(logits, scores, n, finished, pad, eos)
    B, K, V = logits.shape
    n = n or K
    ref = reference(logits, scores, n, finished, pad)
    gs, gp, gt = (got[k].cpu().numpy() for k in ("scores", "parents", "tokens"))
    assert gs.shape == gp.shape == gt.shape == (B, n)
    for b, (sc, be, to) in enumerate(ref):
        want = sc[:n]
        fin = np.isfinite(want)
        assert (np.isfinite(gs[b]) == fin).all() and (gs[b][~fin] == want[~fin]).all(), (b, gs[b], want)
        assert (np.abs(gs[b][fin] - want[fin]) <= U32 * np.abs(want[fin]) + E_LSE).all(), (b, gs[b], want)
        bad = (gp[b] != be[:n]) | (gt[b] != to[:n])
        for r in np.nonzero(bad)[0]:
            assert not exact and fin[r]
            near = np.nonzero((be == gp[b, r]) & (to == gt[b, r]))[0]
            assert len(near) and abs(sc[near[0]] - sc[r]) <= 2 * E_LSE, (b, r, gp[b, r], gt[b, r], be[r], to[r])
    if eos is not None:
        f = got["finished"].cpu().numpy()
        was = np.zeros((B, K), bool) if finished is None else finished.cpu().numpy()
        assert (f == (np.take_along_axis(was, gp, 1) | (gt == eos))).all()
    return got


def head(B, K, V, seed, dtype="bf16", std=2.0):
    z = normal((B, K, V), seed, std=std)
    likely = normal((B, K, V), seed + 1) > 3.0
    return (z + 6.0 * likely).to(DTYPES[dtype]), -normal((B, K), seed + 2, std=3.0).abs()


@pytest.mark.parametrize("B,K,V,n", [(1, 1, 1, 1), (1, 4, 3, 8), (1, 4, 37, 8), (2, 3, 8192, 3), (3, 2, 8193, 4),
                                     (1, 4, 32768, 8), (2, 5, 50257, 10), (4, 4, 151936, 8), (1, 64, 100, 64),
                                     (70, 2, 1000, 2), (1, 1, 300001, 64), (300, 3, 4097, 5), (1, 33, 16384, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_sizes(B, K, V, n, dtype):
    z, s = head(B, K, V, B + K + V, dtype)
    check(z, s, n, eos=int(V // 2))


@pytest.mark.parametrize("V,n", [(30011, 16), (30011, 4), (24576, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("order", ["random", "up", "down"])
def test_parts_of_many_chunks(V, n, dtype, order):
    """So many rows that a block goes through several chunks of one, with candidates in all of them, in the last
    or in the first."""
    z, s = head(160, 4, V, V + n, dtype)
    if order != "random":
        z = z.sort(dim=-1, descending=order == "down").values
    check(z[::16], s[::16], n)                    # few rows: many parts
    from lm_head_linear_chunked_gb300.beam import beam_select
    all_rows = beam_select(z, s, n)
    few = beam_select(z[::16], s[::16], n)
    near = 2 * E_LSE
    for k in ("tokens", "parents"):
        same = (all_rows[k][::16] == few[k])
        gap = (all_rows["scores"][::16, 1:] - all_rows["scores"][::16, :-1]).abs() <= near
        tied = torch.zeros_like(same)
        tied[:, 1:] |= gap
        tied[:, :-1] |= gap
        assert bool((same | tied).all()), k
    check(z[:152:19].contiguous(), s[:152:19], n)
    assert (all_rows["scores"][::16] - few["scores"]).abs().max() <= near


@pytest.mark.parametrize("V", [50, 8200, 33333, 65536])
@pytest.mark.parametrize("n", [1, 7, 64])
def test_equal_logits(V, n):
    """Constant rows and rows of few values: the lower token, and the lower beam, first."""
    K = 3
    z = torch.zeros((1, K, V), device="cuda")
    s = torch.zeros((1, K), device="cuda")
    check(z, s, n, exact=True)
    z[0, 1] = 5.0
    z[0, 2] = normal((V,), V).round()
    s[0] = torch.tensor([0.0, 1.0, 30.0])  # no two beams near each other
    check(z.to(torch.bfloat16), s, n, exact=True)


@pytest.mark.parametrize("V", [40961, 50257])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_equal_beams(V, dtype):
    """The same row at other alignments: equal sums, so the lower beam wins every tie."""
    z, s = head(2, 1, V, 71, dtype)
    z, s = z.expand(2, 5, V).contiguous(), s.expand(2, 5).contiguous()
    check(z, s, 12, exact=True)


@pytest.mark.parametrize("kind", ["up", "down", "lanes", "one thread", "steps"])
@pytest.mark.parametrize("n", [4, 64])
def test_rows_that_fill_the_candidates(kind, n):
    """Orders and places that pass many elements on: rising rows, rows whose large values lie with few threads."""
    V = 30000
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    z = {"up": i / 1000, "down": -i / 1000, "lanes": ((i // 4) % 32 < 16) * 20.0 + (i * 7919 % 4999) / 1000,
         "one thread": ((i // 4) % 256 == 77) * 20.0 + (i * 7919 % 4999) / 1000,
         "steps": (i // 8192) * 10 + (i * 7919 % 4999) / 1000}[kind].view(1, 1, V)
    s = torch.zeros((1, 1), device="cuda")
    check(z, s, n, exact=True)
    check(z.to(torch.bfloat16), s, n, exact=True)


def test_masked_and_bad_logits():
    z, s = head(3, 4, 9001, 83, "fp32")
    z[:, :, normal((9001,), 84) > -1.0] = -float("inf")
    z[0, 1] = -float("inf")                       # nothing left
    z[1, 2, :] = -float("inf")
    z[1, 2, 8500] = 1.5                           # one token left
    z[2, 0, 17] = float("nan")
    z[2, 1, 4000:4003] = float("inf")
    z[2, 3] = float("nan")
    got = check(z, s, 6)
    assert not torch.isnan(got["scores"]).any()
    z[:] = -float("inf")                          # no token anywhere
    from lm_head_linear_chunked_gb300.beam import beam_select
    got = beam_select(z, s, 6)
    assert torch.isinf(got["scores"]).all() and bool((got["scores"] < 0).all())
    assert torch.equal(got["tokens"], torch.arange(6, device="cuda").expand(3, 6)) and not got["parents"].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_the_lowest_value_of_the_type_as_a_mask(dtype):
    z, s = head(2, 3, 5000, 89, dtype)
    z[:, :, 100:] = torch.finfo(DTYPES[dtype]).min
    check(z, s, 5)
    z[0] = torch.finfo(DTYPES[dtype]).min
    check(z, s, 5)


def test_dead_and_finished_beams():
    z, s = head(4, 4, 3000, 97)
    s[0, 1:] = -float("inf")                      # the first step: one live beam
    s[1] = -float("inf")
    s[2, 2] = float("nan")
    finished = torch.zeros((4, 4), dtype=torch.bool, device="cuda")
    check(z, s, 8, finished, pad=9, eos=3)
    finished[0, 0] = finished[2, 1] = finished[3, 0] = finished[3, 3] = True
    z[3, 0] = float("nan")                        # a finished beam's logits are not read
    check(z, s, 8, finished, pad=9, eos=3)
    finished[:] = True
    check(z, s, 8, finished, pad=9, eos=3, exact=True)


def test_logits_of_a_last_position_and_a_wider_row():
    from lm_head_linear_chunked_gb300.beam import beam_select
    z, s = head(6, 3, 1000, 101)
    ref = beam_select(z, s, 5)
    long = torch.zeros((6, 3, 4, 1000), dtype=z.dtype, device="cuda")
    long[:, :, -1] = z
    wide = torch.zeros((6, 3, 1007), dtype=z.dtype, device="cuda")
    wide[:, :, 3:1003] = z
    turned = z.transpose(0, 1).contiguous().transpose(0, 1)
    for v in (long[:, :, -1], wide[:, :, 3:1003], turned):
        got = beam_select(v, s.T.contiguous().T, 5)
        assert all(torch.equal(got[k], ref[k]) for k in ref)


def test_side_stream_and_graph_capture():
    from lm_head_linear_chunked_gb300.beam import beam_reorder, beam_select
    z, s = head(2, 4, 32768, 103)
    cache = normal((8, 2, 33, 16), 104, torch.bfloat16)
    other = torch.empty_like(cache)
    ref = beam_select(z, s, eos_token=5)
    want = beam_reorder([cache], ref["parents"])[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = beam_select(z, s, eos_token=5)
        moved = beam_reorder([cache], got["parents"])[0]
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], ref[k]) for k in ref) and torch.equal(moved, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = beam_select(z, s, eos_token=5)
        beam_reorder([cache], out["parents"], out=[other])
    for _ in range(2):
        other.zero_()
        for k in out:
            out[k].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], ref[k]) for k in ref) and torch.equal(other, want)


# ---------------------------------------------------------------- states

def moved(x, parents):
    B, n = parents.shape
    k = x.shape[0] // B
    rows = (parents + torch.arange(B, device=parents.device)[:, None] * k).reshape(-1)
    return x[rows]


@pytest.mark.parametrize("B,K,n", [(1, 1, 1), (2, 4, 4), (3, 2, 5), (1, 5, 2), (40, 3, 3)])
def test_states_of_every_type_and_shape(B, K, n):
    from lm_head_linear_chunked_gb300.beam import beam_reorder
    g = torch.Generator(device="cuda").manual_seed(B)
    parents = torch.randint(K, (B, n), device="cuda", generator=g)
    R = B * K
    states = [normal((R, 3, 17, 8), 1, torch.bfloat16), normal((R, 7), 2), torch.randint(1 << 40, (R, 129), device="cuda"),
              normal((R,), 3, torch.float16), (normal((R, 5, 3), 4) > 0), normal((R, 0, 4), 5),
              torch.randint(256, (R, 4099), device="cuda").to(torch.uint8), normal((R, 2, 9000), 6, torch.bfloat16)]
    got = beam_reorder(states, parents, check=True)
    for x, y in zip(states, got):
        assert y.is_contiguous() and torch.equal(y, moved(x, parents))


def test_many_states():
    from lm_head_linear_chunked_gb300.beam import beam_reorder
    parents = torch.tensor([[1, 1, 0], [2, 0, 2]], device="cuda")
    states = [normal((6, i % 5 + 1, 8), i) for i in range(61)]
    for x, y in zip(states, beam_reorder(states, parents)):
        assert torch.equal(y, moved(x, parents))


def test_the_used_part_of_caches():
    """Views into caches with room to grow: only the used part moves, into views of the second set."""
    from lm_head_linear_chunked_gb300.beam import beam_reorder
    parents = torch.tensor([[3, 0, 0, 1], [2, 2, 1, 3]], device="cuda")
    for length in (1, 5, 40):
        cache = [normal((8, 2, 40, 16), 7 + i, torch.bfloat16) for i in range(4)]
        other = [torch.full_like(c, -7.0) for c in cache]
        got = beam_reorder([c[:, :, :length] for c in cache], parents, out=[o[:, :, :length] for o in other])
        for c, o, y in zip(cache, other, got):
            assert y.data_ptr() == o.data_ptr()
            assert torch.equal(o[:, :, :length], moved(c[:, :, :length], parents))
            assert bool((o[:, :, length:] == -7.0).all())


def test_odd_strides():
    from lm_head_linear_chunked_gb300.beam import beam_reorder
    parents = torch.tensor([[1, 0]], device="cuda")
    base = normal((2, 6, 7, 9, 11), 11)
    views = [base[:, 1:4, 2:5, ::3], base.transpose(1, 4), base[..., 1:], base[:, :, 3, 4, 5], base[:, ::2, ::2, ::2, ::2]]
    for v, y in zip(views, [beam_reorder([v], parents)[0] for v in views]):
        assert torch.equal(y, moved(v, parents))


def test_a_bad_parent_gives_zeros_and_is_reported():
    from lm_head_linear_chunked_gb300.beam import beam_reorder
    x = normal((4, 33), 13) + 100
    parents = torch.tensor([[1, 2], [-1, 0]], device="cuda")
    y = beam_reorder([x], parents)[0]
    assert torch.equal(y[0], x[1]) and torch.equal(y[3], x[2]) and not y[1].any() and not y[2].any()
    with pytest.raises(lce.LCEError) as e:
        beam_reorder([x], parents, check=True)
    assert e.value.status == 8


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes."""
    from lm_head_linear_chunked_gb300.beam import beam_reorder
    x = torch.empty((5, 1 << 30), dtype=torch.uint8, device="cuda")
    for i in range(5):
        x[i] = i + 1
    y = beam_reorder([x], torch.tensor([[4, 0, 3, 4, 2]], device="cuda"))[0]
    for i, want in enumerate((5, 1, 4, 5, 3)):
        assert int(y[i].min()) == int(y[i].max()) == want


def select_into(z, s, n, finished=None, pad=0):
    """beam_select through the C ABI into outputs filled beforehand: a result that is not written shows."""
    B, K, V = z.shape
    code = {torch.bfloat16: lce.BF16, torch.float16: lce.F16, torch.float32: lce.F32}[z.dtype]
    scores = torch.full((B, n), 12345.0, device="cuda")
    tokens, parents = (torch.full((B, n), -77, dtype=torch.int64, device="cuda") for _ in range(2))
    size = lce.lce_beam_workspace_size(B, K, V, n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    lce.lce_beam_select(B, K, V, n, code, z, V, s, finished, pad, -1, scores, tokens, parents, None, ws, size,
                        torch.cuda.current_stream())
    return {"scores": scores, "tokens": tokens, "parents": parents}


@pytest.mark.parametrize("K,n", [(1, 1), (1, 4), (4, 4), (1, 64), (4, 64), (5, 64), (64, 64)])  # K n on both sides of 256
@pytest.mark.parametrize("V", [100, 600, 9001, 32768, 50257])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_an_item_of_nan_alone(K, n, V, dtype):
    """NaN counts as -inf: scores of -inf, the lowest tokens of the first beam."""
    z = torch.full((2, K, V), float("nan"), dtype=DTYPES[dtype], device="cuda")
    s = torch.zeros((2, K), device="cuda")
    got = select_into(z, s, n)
    assert torch.isneginf(got["scores"]).all() and not got["parents"].any()
    assert torch.equal(got["tokens"], torch.arange(n, device="cuda").expand(2, n))
    # the second beam alone is alive
    if K > 1:
        z[:, 1] = torch.linspace(-3, 3, V, device="cuda")
        check(z, s, n, exact=True)


@pytest.mark.parametrize("rows", [1, 160])  # a row in many parts, and in one
@pytest.mark.parametrize("n", [1, 8, 64])
@pytest.mark.parametrize("V", [700, 9001, 24576])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_nan_and_minus_infinity_beside_few_tokens(rows, n, V, dtype):
    """Fewer finite logits than results: what follows them goes by the token, NaN and -inf alike."""
    z = torch.full((rows, 4, V), -float("inf"), dtype=DTYPES[dtype], device="cuda")
    z[normal(z.shape, 131) > 0] = float("nan")
    for k, at in enumerate((0, V // 3, V // 2, V - 1)):
        z[:, k, at] = 0.5 * k
    z[:, 3, :at // 2] = float("nan")
    s = torch.tensor([0.0, -4.0, -8.0, -12.0], device="cuda").expand(rows, 4).contiguous()
    check(z[:2], s[:2], n, exact=True)
    got, want = select_into(z, s, n), select_into(z[:1].contiguous(), s[:1].contiguous(), n)
    assert all(torch.equal(got[k][:1], want[k]) for k in want)


@pytest.mark.parametrize("d", [1, 2, 3, 4])
def test_both_sets_of_states_in_one_buffer(d):
    from lm_head_linear_chunked_gb300.beam import beam_reorder
    shape = [6, 4, 3, 5]
    shape.insert(d, 2)
    both = normal(tuple(shape), 17)
    parents = torch.tensor([[2, 0, 1], [1, 1, 2]], device="cuda")
    a, b = both.unbind(d)
    before, want = a.clone(), moved(a, parents)
    beam_reorder([a], parents, out=[b])
    assert torch.equal(a, before) and torch.equal(b, want)


def test_conjugate_and_negative_views_as_states():
    """Views whose memory stands for other values."""
    from lm_head_linear_chunked_gb300.beam import beam_reorder
    z = torch.complex(normal((6, 4), 18), normal((6, 4), 19))
    parents = torch.tensor([[2, 0, 1], [1, 1, 2]], device="cuda")
    for x in (z.conj(), z.conj().imag, z.imag):
        assert torch.equal(beam_reorder([x], parents)[0], moved(x, parents))
        out = torch.empty_like(x.resolve_conj().resolve_neg())
        beam_reorder([x], parents, out=[out])
        assert torch.equal(out, moved(x, parents))
