"""Embedding on the GPU: the lookup bit by bit, its gradient against float64."""
import pytest
import torch

from tests.op_util import DTYPES, U32, assert_within, half_step, normal, tiny
from tests.row_refs import embedding_grad_ref

pytestmark = pytest.mark.gpu


def tokens_of(kind, N, V, seed=0, dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "one":
        t = torch.full((N,), V // 2, device="cuda")
    elif kind == "distinct":
        t = torch.randperm(max(N, V), device="cuda", generator=g)[:N] % V
    elif kind == "few":  # long runs beside single tokens
        t = torch.where(torch.rand(N, device="cuda", generator=g) < 0.5, V - 1, torch.randint(V, (N,), device="cuda", generator=g))
    else:  # Zipf: many of a few, few of many
        p = torch.arange(1, V + 1, dtype=torch.float64, device="cuda") ** -1.1
        t = torch.searchsorted(p.cumsum(0) / p.sum(), torch.rand(N, dtype=torch.float64, device="cuda", generator=g)).clamp(max=V - 1)
    return t.to(dtype)


def check_grad(got, dy, tokens, V, scale, padding=None, before=None):
    """FP32 sums of n terms in any order are off by n U32 of the sum of magnitudes; scaling and adding by U32 each."""
    ref, each, n = embedding_grad_ref(dy, tokens, V, scale, padding)
    tol = (n[:, None] + 4) * U32 * each
    if before is not None:
        ref, tol = ref + before.double(), tol + 2 * U32 * before.double().abs()
    assert_within(got, ref, tol + ref.abs() * half_step(got.dtype) + tiny(got.dtype), "grad_weight")
    if before is None:
        assert not got[n == 0].any()  # exactly zero
    else:
        assert torch.equal(got[n == 0], before[n == 0])


@pytest.mark.parametrize("H", [1, 3, 8, 64, 200, 1024, 1601, 4096, 5000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_lookup(H, dtype):
    from lm_head_linear_chunked_gb300.embedding import embedding
    V = 333
    w = normal((V, H), 1, DTYPES[dtype])
    for N, index, scale in ((1, torch.int32, 1.0), (77, torch.int64, 3.7), (1030, torch.int32, 0.02)):
        t = tokens_of("zipf", N, V, 2, index)
        y = embedding(t, w, scale)
        assert torch.equal(y, (w[t.long()].float() * torch.tensor(scale, device="cuda")).to(w.dtype))
    wide = normal((V, H + 9), 3, DTYPES[dtype])  # rows further apart, off vectors' boundaries
    for cut in (slice(0, H), slice(8, 8 + H), slice(1, 1 + H)):
        t = tokens_of("few", 200, V, 4).view(2, 100)
        y = embedding(t, wide[:, cut])
        assert y.shape == (2, 100, H) and torch.equal(y, wide[:, cut][t])
    assert embedding(torch.empty((0, 3), dtype=torch.int64, device="cuda"), w).shape == (0, 3, H)
    assert torch.equal(embedding(torch.tensor(5, device="cuda"), w), w[5])


def test_padding_and_tokens_outside():
    import lm_head_linear_chunked_gb300 as lce
    from lm_head_linear_chunked_gb300.embedding import embedding, embedding_backward
    V = 40
    for H in (64, 65):
        w = normal((V, H), 5)
        t = torch.tensor([3, 7, -1, V, 7, -100, V - 1, 2**31, -2**31, 0], device="cuda")
        y = embedding(t, w, 2.0, -100)
        for i, v in enumerate(t.tolist()):
            if v == -100:
                assert not y[i].any()
            elif 0 <= v < V:
                assert torch.equal(y[i], 2 * w[v])
            else:
                assert bool(y[i].isnan().all())
        assert torch.equal(embedding(t[:2], w, 1.0, 7)[1], w[7])  # padding inside: its row
        dy = normal((10, H), 6)
        check_grad(embedding_backward(dy, t, V, 2.0, -100), dy, t, V, 2.0, -100)
        check_grad(embedding_backward(dy, t, V, 2.0, 7), dy, t, V, 2.0, 7)
        for call in (lambda t: embedding(t, w, 1.0, -100, check=True), lambda t: embedding_backward(dy, t, V, 1.0, -100, check=True)):
            with pytest.raises(lce.LCEError) as e:
                call(t)
            assert e.value.status == 8
            call(torch.where((t < V) & (t >= 0), t, -100))  # fine without them
            call(torch.where((t < V) & (t >= 0), t, -100).int())
        # a dy that is not finite stays with its token
        dy[0, 0], dy[4, 1] = float("nan"), float("inf")
        grad = embedding_backward(dy, t, V, 1.0, -100)
        assert int((~grad.isfinite()).sum()) == 2 and bool(grad[3, 0].isnan()) and not bool(grad[7, 1].isfinite())


@pytest.mark.parametrize("N,V,H", [(0, 5, 8), (1, 1, 1), (2, 1, 64), (31, 97, 33), (33, 1023, 64), (1000, 1024, 200), (1025, 1025, 256),
                                   (5000, 50257, 64), (3000, 151936, 128), (20000, 300, 1601), (70000, 151936, 40),
                                   (2000, (1 << 20) + 3, 8), (4097, 7, 4096), (6144, 3000, 24), (6145, 60000, 24), (513, 2000, 5000), (300000, 5000, 16)])
@pytest.mark.parametrize("kind", ["one", "distinct", "few", "zipf"])
def test_gradient(N, V, H, kind):
    from lm_head_linear_chunked_gb300.embedding import embedding_backward
    for dtype, gtype in (("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")):
        t = tokens_of(kind, N, V, 7, torch.int32 if H % 16 else torch.int64)
        dy = normal((N, H), 8, DTYPES[dtype])
        got = embedding_backward(dy, t, V, 1.25, None, DTYPES[gtype])
        check_grad(got, dy, t, V, 1.25)
        assert torch.equal(got, embedding_backward(dy, t, V, 1.25, None, DTYPES[gtype]))  # equal calls, equal bits
        if V * H > 1 << 24:
            break


@pytest.mark.parametrize("H", [64, 200, 1601, 4096])
def test_outputs_given_and_added_to(H):
    from lm_head_linear_chunked_gb300.embedding import embedding_backward
    V, N = 500, 3000
    t = tokens_of("few", N, V, 9)
    t[t < 250] = 3
    for dtype in (torch.bfloat16, torch.float32):
        dy = normal((N, H), 10, dtype)
        for room in (H, H + 8, H + 3):
            acc = normal((V, room), 11)
            before = acc.clone()
            out = embedding_backward(dy, t, V, 0.5, V - 1, out=acc[:, :H], accumulate=True)
            assert out.data_ptr() == acc.data_ptr()
            check_grad(out, dy, t, V, 0.5, V - 1, before[:, :H])
            assert torch.equal(acc[:, H:], before[:, H:])
            out = embedding_backward(dy, t, V, 0.5, V - 1, out=acc[:, :H])
            check_grad(out, dy, t, V, 0.5, V - 1)
            assert torch.equal(acc[:, H:], before[:, H:])
        wide = normal((N, H + 5), 12, dtype)
        for cut in (slice(0, H), slice(5, 5 + H)):
            check_grad(embedding_backward(wide[:, cut], t, V), wide[:, cut], t, V, 1.0)
        check_grad(embedding_backward(dy[:1].expand(N, H), t, V), dy[:1].expand(N, H), t, V, 1.0)


@pytest.mark.parametrize("N", [1, 3, 31, 33, 63, 255, 256, 257])
@pytest.mark.parametrize("H", [1, 64, 513, 4096])
def test_few_tokens(N, H):
    """A short path to 256 tokens: into a new gradient, one given and one that has values, which other rows keep."""
    from lm_head_linear_chunked_gb300.embedding import embedding_backward
    V = 700
    for kind in ("one", "distinct", "few"):
        t = tokens_of(kind, N, V, 21)
        if N > 4:
            t[2], t[3], t[4] = -100, V, -5
        for dtype in (torch.bfloat16, torch.float16, torch.float32):
            dy = normal((N, H), 22, dtype)
            check_grad(embedding_backward(dy, t, V, 0.5, -100), dy, t, V, 0.5, -100)
            acc = normal((V, H + 3), 23)
            before = acc.clone()
            out = embedding_backward(dy, t, V, 0.5, -100, out=acc[:, :H], accumulate=True)
            check_grad(out, dy, t, V, 0.5, -100, before[:, :H])
            unnamed = torch.ones(V, dtype=torch.bool, device="cuda")
            unnamed[t[(t >= 0) & (t < V)]] = False
            assert torch.equal(out[unnamed], before[:, :H][unnamed]) and torch.equal(acc[:, H:], before[:, H:])
            check_grad(embedding_backward(dy, t, V, 0.5, -100, out=acc[:, :H]), dy, t, V, 0.5, -100)


@pytest.mark.parametrize("H", [1, 2, 3, 63, 128, 129, 255, 256, 257, 258, 511, 1601])
@pytest.mark.parametrize("start", [0, 1, 2, 3])
def test_16_bit_rows_on_any_boundary(H, start):
    """Gradients that start anywhere, side by side or apart, with NaN before, between and behind them."""
    from lm_head_linear_chunked_gb300.embedding import embedding_backward
    V = 90
    for N, kind in ((300, "one"), (1000, "few"), (7001, "zipf")):
        t = tokens_of(kind, N, V, 27)
        for gap in (0, 1, 5):
            for dtype in (torch.bfloat16, torch.float16):
                flat = torch.full((start + N * (H + gap) + 8,), float("nan"), device="cuda", dtype=dtype)
                dy = flat[start:start + N * (H + gap)].view(N, H + gap)[:, :H]
                dy.copy_(normal((N, H), 28, dtype))
                check_grad(embedding_backward(dy, t, V, 0.5, 3), dy, t, V, 0.5, 3)
                acc = normal((V, H + 1), 29)
                before = acc.clone()
                check_grad(embedding_backward(dy, t, V, 0.5, 3, out=acc[:, 1:], accumulate=True), dy, t, V, 0.5, 3, before[:, 1:])
                assert torch.equal(acc[:, 0], before[:, 0])


def test_an_output_that_autograd_has_saved():
    """Written into, it is not what was saved: the backward that would read it says so."""
    from lm_head_linear_chunked_gb300.embedding import embedding_backward
    t, dy = tokens_of("zipf", 40, 30, 24), normal((40, 16), 25)
    acc, x = torch.zeros(30, 16, device="cuda"), normal((30, 16), 26).requires_grad_(True)
    y = (x * acc).sum()
    embedding_backward(dy, t, 30, out=acc, accumulate=True)
    with pytest.raises(RuntimeError, match="modified"):
        y.backward()
    with torch.inference_mode():
        acc = torch.zeros(30, 16, device="cuda")
        check_grad(embedding_backward(dy, t, 30, out=acc, accumulate=True), dy, t, 30, 1.0)


def test_autograd_and_tied_weights():
    """The module's gradient, and the sum of both uses of a matrix that the head shares."""
    import lm_head_linear_chunked_gb300 as lce
    from lm_head_linear_chunked_gb300.chunk_loss import linear_cross_entropy
    from lm_head_linear_chunked_gb300.embedding import Embedding, embedding_backward
    V, H = 512, 128
    m = Embedding(V, H, 2.0, 9, device="cuda", dtype=torch.bfloat16)
    t = tokens_of("zipf", 300, V, 13).view(3, 100)
    c = normal((3, 100, H), 14, torch.bfloat16)
    grad = torch.autograd.grad(m(t), m.weight, c)[0]
    assert torch.equal(grad, embedding_backward(c, t, V, 2.0, 9))
    assert not m(t.detach()).detach().requires_grad
    m(t).sum().backward()  # an expanded gradient
    assert torch.equal(m.weight.grad, embedding_backward(torch.ones_like(c), t, V, 2.0, 9))
    # tied: autograd adds the two parts; by hand they go into one float32 accumulator
    labels = t.roll(-1, 1)
    h = normal((300, H), 15, torch.bfloat16)
    w = m.weight.detach()
    out = lce.fused(h, w, None, labels.reshape(-1))
    head = out["grad_W_acc"].clone()
    embedding_backward(c, t, V, 2.0, 9, out=out["grad_W_acc"], accumulate=True)
    check_grad(out["grad_W_acc"], c, t, V, 2.0, 9, head)
    m.weight.grad = None
    (linear_cross_entropy(h, m.weight, labels.reshape(-1)) + (m(t) * c).float().sum()).backward()
    both = out["grad_W_acc"].double()
    parts = head.abs().double() + embedding_grad_ref(c, t, V, 2.0, 9)[0].abs()
    assert_within(m.weight.grad, both, 3 * half_step(torch.bfloat16) * parts + 1e-6, "tied gradient")  # three roundings to bf16


def check_named(got, dy, tokens, V, scale):
    """As check_grad, over the rows that tokens name alone; the others have to be zero (got is cleared)."""
    tokens = tokens.reshape(-1)
    inside = (tokens >= 0) & (tokens < V)
    named, at = tokens[inside].unique(return_inverse=True)
    check_grad(got[named], dy[inside], at, named.numel(), scale)
    got[named] = 0
    assert not got.any()


@pytest.mark.parametrize("N", [0, 1, 33])
@pytest.mark.parametrize("H,dtype", [(4096, "bf16"), (1024, "fp32")])
@pytest.mark.parametrize("gap", [0, 3])
def test_few_tokens_into_a_large_gradient(N, H, dtype, gap):
    """Every row is written, above the half gigabyte that is cleared beside the sort as below it."""
    from lm_head_linear_chunked_gb300.embedding import embedding_backward
    V = 151936
    room = torch.full((V, H + gap), float("nan"), device="cuda", dtype=DTYPES[dtype])
    t, dy = tokens_of("few", N, V, 31), normal((N, H), 32, DTYPES[dtype])
    got = embedding_backward(dy, t, V, 0.5, out=room[:, :H])
    check_named(got, dy, t, V, 0.5)
    assert bool(room[:, H:].isnan().all())


@pytest.mark.parametrize("N,V,H", [(50, 300, 64), (3000, 5000, 65), (9000, 9001, 33)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_an_output_beside_the_gradient(N, V, H, dtype):
    """Both are columns of one buffer; neither reaches into the other."""
    from lm_head_linear_chunked_gb300.embedding import embedding_backward
    both = normal((V, 2 * H + 1), 33, DTYPES[dtype])
    before, t = both.clone(), tokens_of("few", N, V, 34)
    got = embedding_backward(both[:N, H:2 * H], t, V, 0.5, out=both[:, :H])
    check_grad(got, before[:N, H:2 * H], t, V, 0.5)
    assert torch.equal(both[:, H:], before[:, H:])
