"""The operators between token ids and the head as a program uses them: through the C ABI with buffers of its own,
captured and replayed, on other streams, beyond 2^32 bytes, and all of them in one model."""
import pytest
import torch

import lm_head_linear_chunked_gb300 as lce
from tests.op_util import U32, assert_within, normal
from tests.row_refs import embedding_grad_ref
from tests.test_gpu_embedding import tokens_of
from tests.test_gpu_expert_rows import experts_of
from tests.test_gpu_operators_abi import Buffers, stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,H", [(5, 1), (300, 1601), (1000, 2560), (77, 512), (3, 40000), (9, 16384)])
def test_rms_norm_abi(rows, H):
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_backward, rms_norm_forward, rms_norm_fp8
    x, r, dy, ds = (normal((rows, H), k, torch.bfloat16) for k in range(4))
    w = normal(H, 5)
    B = Buffers()
    y, s, dx = (B.take((rows, H), torch.bfloat16) for _ in range(3))
    rstd, dw = B.take((rows,), torch.float32), B.take((H,), torch.float32)
    q, scales = B.take((rows, H), torch.uint8), B.take((rows, -(-H // 128)), torch.float32)
    nws = lce.lce_rms_norm_workspace_size(rows, H)
    ws = B.take((nws,), torch.uint8)
    lce.lce_rms_norm_forward(rows, H, lce.BF16, lce.F32, x, H, r, H, w, 1e-5, s, H, y, H, rstd, stream())
    lce.lce_rms_norm_backward(rows, H, lce.BF16, lce.F32, dy, H, s, H, w, rstd, ds, H, dx, H, dw, ws, nws, stream())
    f = rms_norm_forward(x, w, r, 1e-5)
    d = rms_norm_backward(dy, f["sum"], w, f["rstd"], ds)
    for got, want in ((y, f["y"]), (s, f["sum"]), (rstd, f["rstd"]), (dx, d["grad_x"]), (dw, d["grad_weight"])):
        assert torch.equal(got, want)
    lce.lce_rms_norm_fp8(rows, H, lce.BF16, lce.F32, x, H, r, H, w, 1e-5, s, H, q, H, scales, lce.FP8_GROUP, stream())
    B.check()
    e = rms_norm_fp8(x, w, r, 1e-5)
    assert torch.equal(q, e["q"].view(torch.uint8)) and torch.equal(scales, e["scales"])


@pytest.mark.parametrize("N,V,H", [(1, 1, 1), (33, 7, 96), (700, 1500, 201), (5000, 300, 512), (5000, 90000, 128), (200, 40, 4096)])
@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, lce.BF16), (torch.float32, lce.F32)])
def test_embedding_abi(N, V, H, dtype, code):
    from lm_head_linear_chunked_gb300.embedding import embedding, embedding_backward
    t, w, dy = tokens_of("few", N, V, 1), normal((V, H), 2, dtype), normal((N, H), 3, dtype)
    B = Buffers()
    y, dw = B.take((N, H), dtype), B.take((V, H), dtype)
    acc = B.take((V, H), torch.float32)
    nws = lce.lce_embedding_workspace_size(N, V, H)
    ws = B.take((nws,), torch.uint8)
    lce.lce_embedding_forward(N, V, H, code, t, 8, w, H, 0.5, lce.NO_PADDING, y, H, None, stream())
    lce.lce_embedding_backward(N, V, H, code, code, t, 8, dy, H, 0.5, V - 1, dw, H, ws, nws, stream(), 0)
    assert lce.lce_check_status(ws, stream()) == 0
    B.check()
    assert torch.equal(y, embedding(t, w, 0.5)) and torch.equal(dw, embedding_backward(dy, t, V, 0.5, V - 1))
    acc.copy_(normal((V, H), 4))
    want = embedding_backward(dy, t, V, 0.5, V - 1, out=acc.clone(), accumulate=True)
    lce.lce_embedding_backward(N, V, H, code, lce.F32, t, 8, dy, H, 0.5, V - 1, acc, H, ws, nws, stream(), lce.ACCUMULATE)
    B.check()
    assert torch.equal(acc, want)


@pytest.mark.parametrize("T,k,E,H,align", [(1, 1, 1, 1, 1), (40, 2, 8, 64, 1), (700, 3, 61, 201, 16), (3000, 8, 128, 96, 128), (50, 8, 9, 4096, 4)])
def test_expert_rows_abi(T, k, E, H, align):
    from lm_head_linear_chunked_gb300.expert_rows import combine, combine_backward, dispatch, dispatch_backward, expert_plan
    experts, mask = experts_of(T, k, E, 1, "unused"), normal((T,), 2) > -1
    R = lce.lce_expert_rows(T, k, E, align)
    B = Buffers()
    pos, slots = B.take((T, k), torch.int32), B.take((R,), torch.int32)
    counts, offsets = B.take((E,), torch.int64), B.take((E + 1,), torch.int64)
    nws = lce.lce_expert_plan_workspace_size(T, k, E)
    ws = B.take((nws,), torch.uint8)
    lce.lce_expert_plan(T, k, E, align, experts, 8, mask, pos, slots, counts, offsets, ws, nws, stream())
    assert lce.lce_check_status(ws, stream()) == 0
    plan = expert_plan(experts, E, mask, align)
    for got, name in ((pos, "positions"), (slots, "slots"), (counts, "counts"), (offsets, "offsets")):
        assert torch.equal(got, plan[name])
    x, dy, w = normal((T, H), 3, torch.bfloat16), normal((T, H), 4, torch.bfloat16), normal((T, k), 5)
    rows = normal((R, H), 6, torch.bfloat16)
    xs, y, dr, dx = (B.take(s, torch.bfloat16) for s in ((R, H), (T, H), (R, H), (T, H)))
    dw = B.take((T, k), torch.float32)
    lce.lce_expert_dispatch(T, k, H, R, lce.BF16, x, H, pos, slots, xs, H, stream())
    lce.lce_expert_combine(T, k, H, R, lce.BF16, lce.F32, rows, H, w, pos, y, H, stream())
    lce.lce_expert_combine_backward(T, k, H, R, lce.BF16, lce.F32, dy, H, rows, H, w, pos, slots, dr, H, dw, stream())
    lce.lce_expert_dispatch_backward(T, k, H, R, lce.BF16, rows, H, pos, dx, H, stream())
    B.check()
    d = combine_backward(dy, rows, w, plan)
    for got, want in ((xs, dispatch(x, plan)), (y, combine(rows, w, plan)), (dr, d["grad_rows"]), (dw, d["grad_weights"]),
                      (dx, dispatch_backward(rows, plan))):
        assert torch.equal(got, want)


def test_every_kernel_is_seen_and_no_device_memory_is_taken():
    N, V, H = 9000, 4000, 256
    t, dy = tokens_of("zipf", N, V, 1), normal((N, H), 2)
    dw = torch.empty((V, H), device="cuda")
    nws = lce.lce_embedding_workspace_size(N, V, H)
    ws = torch.empty(nws, dtype=torch.uint8, device="cuda")

    def call():
        lce.lce_embedding_backward(N, V, H, lce.F32, lce.F32, t, 8, dy, H, 1.0, lce.NO_PADDING, dw, H, ws, nws, stream(), 0)

    call()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    lce.lce_profile_begin()
    call()
    prof = lce.lce_profile_end()
    assert prof["other"][1] == 6 and prof["other"][0] > 0  # two digits, counted and placed, sums and their end


def operators():
    """name -> (inputs to be refilled, call): each operator on sizes that take several kernels."""
    from lm_head_linear_chunked_gb300.embedding import embedding, embedding_backward
    from lm_head_linear_chunked_gb300.expert_rows import combine, combine_backward, dispatch, dispatch_backward, expert_plan
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_backward, rms_norm_forward, rms_norm_fp8

    def norm(x, r, w, dy):
        f = rms_norm_forward(x, w, r)
        d, e = rms_norm_backward(dy, f["sum"], w, f["rstd"], dy), rms_norm_fp8(x, w, r)
        return f["y"], f["sum"], d["grad_x"], d["grad_weight"], e["q"].view(torch.uint8), e["scales"]

    def lookup(t, w, dy):
        return embedding(t, w, 2.0), embedding_backward(dy, t, w.shape[0], 2.0)

    def experts(x, e, w, dy):
        plan = expert_plan(e, 40, None, 8)
        rows = dispatch(x, plan)
        d = combine_backward(dy, rows, w, plan)
        return (*(plan[k] for k in ("positions", "slots", "counts", "offsets")), rows, combine(rows, w, plan), d["grad_rows"],
                d["grad_weights"], dispatch_backward(d["grad_rows"], plan))

    def inputs(seed):
        b = torch.bfloat16
        return {"norm": (normal((900, 640), seed, b), normal((900, 640), seed + 1, b), normal(640, seed + 2), normal((900, 640), seed + 3, b)),
                "short": (tokens_of("zipf", 700, 900, seed), normal((900, 72), seed, b), normal((700, 72), seed + 1, b)),
                "handful": (tokens_of("zipf", 200, 900, seed), normal((900, 72), seed, b), normal((200, 72), seed + 1, b)),
                "long": (tokens_of("few", 9000, 5000, seed), normal((5000, 136), seed), normal((9000, 136), seed + 1)),
                "sparse": (tokens_of("zipf", 6000, 60000, seed), normal((60000, 24), seed), normal((6000, 24), seed + 1)),
                "experts": (normal((3000, 200), seed, b), experts_of(3000, 4, 40, seed, "unused"), normal((3000, 4), seed + 1),
                            normal((3000, 200), seed + 2, b))}

    return {"norm": norm, "handful": lookup, "short": lookup, "long": lookup, "sparse": lookup, "experts": experts}, inputs


@pytest.mark.parametrize("name", ["norm", "handful", "short", "long", "sparse", "experts"])
def test_side_streams_and_replayed_graphs(name):
    """Two graphs of one operator on their own inputs, replayed in turn and with new inputs, give the eager bits."""
    calls, inputs = operators()
    call = calls[name]
    side = torch.cuda.Stream()
    graphs = []
    for seed in (100, 200):
        mine = inputs(seed)[name]
        want = [t.clone() for t in call(*mine)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = call(*mine)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = call(*mine)
        graphs.append((graph, mine, out))
    for seed in (300, 400, 300):
        new = inputs(seed)[name]
        want = [t.clone() for t in call(*new)]
        for graph, mine, out in graphs:
            for a, b in zip(mine, new):
                a.copy_(b)
            for t in out:
                t.zero_()
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, _, out in graphs:
            for got, w in zip(out, want):
                assert torch.equal(got, w)


def test_rows_beyond_2_to_the_32_bytes():
    from lm_head_linear_chunked_gb300.embedding import embedding, embedding_backward
    from lm_head_linear_chunked_gb300.expert_rows import combine, combine_backward, dispatch, expert_plan
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_backward, rms_norm_forward, rms_norm_fp8
    rows, H = 700000, 4096
    x = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    x[:] = normal((1000, H), 1, torch.bfloat16).repeat(rows // 1000, 1)
    small = x[:1000].clone()
    f, g = rms_norm_forward(x, None, x), rms_norm_forward(small, None, small)
    assert torch.equal(f["y"][-1000:], g["y"]) and torch.equal(f["rstd"][-1000:], g["rstd"]) and torch.equal(f["sum"][-1000:], g["sum"])
    d = rms_norm_backward(x, x, None, f["rstd"], x)["grad_x"]
    assert torch.equal(d[-1000:], rms_norm_backward(small, small, None, g["rstd"], small)["grad_x"])
    del f, d
    e, h = rms_norm_fp8(x), rms_norm_fp8(small)
    assert torch.equal(e["q"][-1000:].view(torch.uint8), h["q"].view(torch.uint8)) and torch.equal(e["scales"][-1000:], h["scales"])
    del e
    # a vocabulary of 5.7 GB, its last rows
    t = rows - 1 - tokens_of("few", 3000, 1000, 2)
    assert torch.equal(embedding(t, x), small[(t - (rows - 1000))])
    dy = normal((3000, H), 3, torch.bfloat16)
    grad = embedding_backward(dy, t, rows)
    ref, each, n = embedding_grad_ref(dy, t - (rows - 1000), 1000, 1.0)
    assert_within(grad[-1000:], ref, (n[:, None] + 4) * U32 * each + ref.abs() * 2.0 ** -8 + 1e-40, "grad_weight")
    assert not grad[:-1000].any()
    del grad
    # 5.2 GB of sorted rows
    T, k, E = 80000, 8, 64
    plan = expert_plan(experts_of(T, k, E, 4), E)
    xs = dispatch(x[:T], plan)
    p = plan["positions"].long()
    assert torch.equal(xs[p[-500:, 7]], x[T - 500:T]) and int(p.max()) == T * k - 1
    y = combine(xs, None, plan)
    assert_within(y[-500:], 8 * x[T - 500:T].double(), x[T - 500:T].double().abs() * 8 * (2.0 ** -8 + 9 * U32) + 1e-40, "y")
    c = combine_backward(x[:T], xs, normal((T, k), 5), plan)
    sq = x[T - 500:T].double().square().sum(1)
    assert_within(c["grad_weights"][-500:], sq[:, None].expand(500, k), (sq * 250 * U32)[:, None].expand(500, k), "grad_weights")


class Model(torch.nn.Module):
    """One mixture block between an embedding and its (tied) head; `plain`: the same in torch's own operations."""

    def __init__(self, dtype, plain, V=300, H=96, E=6):
        super().__init__()
        from lm_head_linear_chunked_gb300.embedding import Embedding
        from lm_head_linear_chunked_gb300.rms_norm import RMSNorm
        self.plain, self.E = plain, E
        self.embedding = Embedding(V, H, H ** 0.5, V - 1, device="cuda", dtype=dtype)
        self.first, self.last = (RMSNorm(H, device="cuda", dtype=dtype) for _ in range(2))
        self.router = torch.nn.Linear(H, E, bias=False, device="cuda", dtype=dtype)
        self.experts = torch.nn.Parameter(torch.empty(E, H, H, device="cuda", dtype=dtype))
        for i, (name, p) in enumerate(self.named_parameters()):
            with torch.no_grad():
                p.copy_(normal(p.shape, 50 + i, std=0.3, mean=1.0 if p.dim() == 1 else 0.0).to(dtype))

    def forward(self, tokens, chosen, align):
        from lm_head_linear_chunked_gb300.expert_rows import combine, dispatch, expert_plan
        if self.plain:
            h = self.embedding.weight[tokens] * self.embedding.scale
            # a row of padding takes no gradient
            h = torch.where((tokens == self.embedding.padding_idx)[..., None], h.detach(), h)
            norm = lambda m, s: s * (s.square().mean(-1, keepdim=True) + m.eps).rsqrt() * m.weight  # noqa: E731
            x = norm(self.first, h)
            share = self.router(x).softmax(-1).gather(-1, chosen)
            work = torch.einsum("bth,ehf->btef", x, self.experts).gather(2, chosen[..., None].expand(*chosen.shape, x.shape[-1]))
            return norm(self.last, (work * share[..., None]).sum(2) + h)
        h = self.embedding(tokens)
        x = self.first(h)
        share = self.router(x).softmax(-1).gather(-1, chosen)
        plan = expert_plan(chosen, self.E, None, align)
        rows = dispatch(x, plan)
        ends = plan["offsets"].tolist()
        work = torch.cat([rows[a:b] @ self.experts[e] for e, (a, b) in enumerate(zip(ends, ends[1:]))] + [rows[ends[-1]:]])
        return self.last(combine(work, share, plan), h)[0]


@pytest.mark.parametrize("align", [1, 16])
def test_a_model_of_them_all(align):
    """fp32 against the same model in float64: six layers whose sums have at most 96 terms (200 tokens for the weights),
    each rounding U32, and gradients that pass all of them twice: 2 x 6 x 200 roundings of the largest value."""
    ours, ref = Model(torch.float32, False), Model(torch.float64, True)
    tokens = tokens_of("zipf", 200, 300, 7).view(4, 50)
    tokens[:, -5:] = 299
    chosen = normal((4, 50, 6), 8).topk(2, dim=-1).indices
    c = normal((4, 50, 96), 9)
    tol = 2 * 6 * 200 * U32
    y, want = ours(tokens, chosen, align), ref(tokens, chosen, align)
    assert_within(y, want.detach(), torch.full_like(want, tol * float(want.detach().abs().max())), "y")
    (y * c).sum().backward()
    (want * c.double()).sum().backward()
    for (name, p), q in zip(ours.named_parameters(), ref.parameters()):
        assert_within(p.grad, q.grad, torch.full_like(q.grad, tol * float(q.grad.abs().max())), name)
    assert not ours.embedding.weight.grad[299].any()


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.filterwarnings("ignore::torch.jit.TracerWarning", "ignore::DeprecationWarning")
def test_a_trace_computes_with_its_own_inputs(grad):
    from lm_head_linear_chunked_gb300.embedding import embedding
    from lm_head_linear_chunked_gb300.expert_rows import combine, dispatch, expert_plan
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm
    plan = expert_plan(experts_of(40, 2, 8, 1), 8)
    w = normal(64, 2)

    def call(x, table):
        y, s = rms_norm(x, w, x)
        return y + 0, s + 0, combine(dispatch(x, plan), None, plan) + 0, embedding(tokens_of("one", 7, 30), table) + 0

    def inputs(seed):
        return tuple(normal(shape, seed).requires_grad_(grad) for shape in ((40, 64), (30, 16)))

    traced = torch.jit.trace(call, inputs(3), check_trace=False)
    for seed in (4, 5):
        a = inputs(seed)
        got, want = traced(*a), call(*a)
        assert all(torch.equal(g, r) for g, r in zip(got, want))
        if grad:
            u, v = (torch.autograd.grad(sum(t.sum() for t in r), a) for r in (got, want))
            assert all(torch.equal(g, r) for g, r in zip(u, v))
