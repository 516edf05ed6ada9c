"""Rows sorted by expert, on the GPU: plans and moves exactly, sums against float64."""
import pytest
import torch

from tests.op_util import DTYPES, U32, assert_within, half_step, normal, tiny
from tests.row_refs import plan_ref, sum_depth

pytestmark = pytest.mark.gpu

PLANS = [(0, 2, 8), (1, 1, 1), (1, 8, 8), (2, 3, 5), (33, 2, 8), (500, 8, 128), (1001, 3, 61), (700, 1, 1024), (130, 6, 1023),
         (4000, 8, 256), (20000, 2, 16)]


def experts_of(T, k, E, seed, kind="any", dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "same":  # every slot names one expert, a token's slots alike
        return torch.full((T, k), E // 2, dtype=dtype, device="cuda")
    e = torch.randint(E, (T, k), device="cuda", generator=g)
    if kind == "unused":
        e[torch.rand(T, k, device="cuda", generator=g) < 0.3] = -1
    return e.to(dtype)


@pytest.mark.parametrize("T,k,E", PLANS)
@pytest.mark.parametrize("align", [1, 16, 128, 1000])
def test_plan(T, k, E, align):
    from lm_head_linear_chunked_gb300.expert_rows import expert_plan
    for kind, dtype, masked in (("any", torch.int64, False), ("unused", torch.int32, True), ("same", torch.int32, False),
                                ("any", torch.int64, True)):
        experts = experts_of(T, k, E, 1, kind, dtype)
        mask = normal((T,), 2) > -0.5 if masked else None
        got = expert_plan(experts, E, mask, align)
        want = plan_ref(experts, E, mask, align)
        for name, w in zip(("positions", "slots", "counts", "offsets"), want):
            assert torch.equal(got[name].cpu(), w), (name, kind)
    if T:
        none = expert_plan(experts, E, torch.zeros(T, dtype=torch.bool, device="cuda"), align)
        assert bool((none["slots"] == -1).all()) and bool((none["positions"] == -1).all()) and not none["offsets"].any()
        three = expert_plan(experts.view(1, T, k), E, None, align)
        assert three["positions"].shape == (1, T, k)


def test_indices_outside():
    import lm_head_linear_chunked_gb300 as lce
    from lm_head_linear_chunked_gb300.expert_rows import expert_plan
    experts = experts_of(3000, 2, 16, 3)
    experts[17, 1], experts[2999, 0], experts[5, 0], experts[6, 0] = 16, -2, 2**40, -2**40
    got = expert_plan(experts, 16, None, 4)
    want = plan_ref(experts, 16, None, 4)
    for name, w in zip(("positions", "slots", "counts", "offsets"), want):
        assert torch.equal(got[name].cpu(), w)
    with pytest.raises(lce.LCEError) as e:
        expert_plan(experts, 16, check=True)
    assert e.value.status == 8
    expert_plan(experts.clamp(-1, 15), 16, check=True)
    left_out = torch.ones(3000, dtype=torch.bool, device="cuda")
    left_out[[17, 2999, 5, 6]] = False
    expert_plan(experts, 16, left_out, check=True)  # nobody looks at a masked token's indices


def refs(x, rows, w, plan):
    """All four moves in float64, and the sums of magnitudes behind each."""
    p = plan["positions"].long()
    has = (p >= 0)[..., None]
    at = p.clamp(min=0)
    got = rows.double()[at] * has
    share = (torch.ones_like(p, dtype=torch.float64) if w is None else w.double()) * has[..., 0]
    return got, share, at, has


def check_moves(T, k, E, H, dtype, wtype, align=1, kind="any", masked=False, seed=0, room=0):
    from lm_head_linear_chunked_gb300.expert_rows import combine, combine_backward, dispatch, dispatch_backward, expert_plan
    t = DTYPES[dtype]
    experts = experts_of(T, k, E, seed + 1, kind)
    mask = normal((T,), seed + 2) > -0.5 if masked else None
    plan = expert_plan(experts, E, mask, align)
    R = plan["slots"].shape[0]
    x = normal((T, H + room), seed + 3, t)[:, room:]
    rows = normal((R, H + room), seed + 4, t)[:, room:]
    dy = normal((T, H + room), seed + 5, t)[:, room:]
    w = normal((T, k), seed + 6, DTYPES[wtype]) if wtype else None
    # rows that no slot takes may hold anything
    rows = torch.where((plan["slots"] >= 0)[:, None], rows, torch.full((), float("nan"), dtype=t, device="cuda"))
    slots = plan["slots"].long()
    token = slots.clamp(min=0) // k
    want = torch.where((slots >= 0)[:, None], x[token] if T else x.new_zeros(R, H), torch.zeros((), dtype=t, device="cuda"))
    assert torch.equal(dispatch(x, plan), want)
    p = plan["positions"].long()
    has = (p >= 0)
    got = torch.where(has[..., None], rows[p.clamp(min=0)].double() if R else torch.zeros(T, k, H, dtype=torch.float64, device="cuda"), 0.0)
    for weights in (w, None):
        share = (torch.ones(T, k, dtype=torch.float64, device="cuda") if weights is None else weights.double()) * has
        y, each = (got * share[..., None]).sum(1), (got * share[..., None]).abs().sum(1)
        tol = each * (k + 1) * U32 + y.abs() * half_step(t) + tiny(t)
        assert_within(combine(rows, weights, plan), y, tol, "y")
        if weights is None:
            assert torch.equal(dispatch_backward(rows, plan), combine(rows, None, plan))
        d = combine_backward(dy, rows, weights, plan)
        flat = share.reshape(-1)[slots.clamp(min=0)] * (slots >= 0) if T else share.new_zeros(R)
        gr = (dy.double()[token] if T else torch.zeros(R, H, dtype=torch.float64, device="cuda")) * flat[:, None]
        assert_within(d["grad_rows"], gr, gr.abs() * (half_step(t) + U32) + tiny(t), "grad_rows")
        assert not d["grad_rows"][slots < 0].any()
        if weights is None:
            assert d["grad_weights"] is None
            continue
        gw, each = (got * dy.double()[:, None]).sum(2), (got * dy.double()[:, None]).abs().sum(2)
        tol = each * (sum_depth(H) + H / 32 + 4) * U32 + gw.abs() * half_step(w.dtype) + tiny(w.dtype)
        assert_within(d["grad_weights"], gw, tol, "grad_weights")
        only = combine_backward(dy, rows, weights, plan, True, False)
        assert only["grad_weights"] is None and torch.equal(only["grad_rows"], d["grad_rows"])
        only = combine_backward(dy, rows, weights, plan, False, True)
        assert only["grad_rows"] is None and torch.equal(only["grad_weights"], d["grad_weights"])


@pytest.mark.parametrize("H", [1, 3, 8, 64, 200, 1024, 1601, 2048, 4096, 8200])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_moves_by_width(H, dtype, wtype):
    check_moves(77, 3, 9, H, dtype, wtype, 4, "unused", True)
    check_moves(5, 1, 2, H, dtype, wtype, 1)


@pytest.mark.parametrize("T,k,E", PLANS)
@pytest.mark.parametrize("align", [1, 128])
def test_moves_by_plan(T, k, E, align):
    check_moves(T, k, E, 72, "bf16", "fp32", align, "unused", True, 10)
    check_moves(T, k, E, 24, "fp32", "fp32", align, "same", False, 20)


@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 16, 17, 40])
def test_moves_by_slots(k):
    check_moves(60, k, 64, 264, "bf16", "bf16", 1, "unused", False, 30)


@pytest.mark.parametrize("room", [1, 2, 4, 8])
@pytest.mark.parametrize("H", [64, 200, 2048, 1601])
def test_strides_and_alignment(room, H):
    check_moves(50, 4, 8, H, "bf16", "fp32", 2, "unused", True, 40, room)
    check_moves(50, 4, 8, H, "fp32", "fp32", 2, "unused", True, 41, room)


def test_a_plan_of_other_rows_reads_nothing_outside():
    """Positions past the rows count as none."""
    from lm_head_linear_chunked_gb300.expert_rows import combine, dispatch, expert_plan
    plan = expert_plan(experts_of(100, 2, 8, 50), 8)
    short = {"positions": plan["positions"], "slots": plan["slots"][:150].contiguous()}
    rows = normal((150, 64), 51)
    y = combine(rows, None, short)
    p = plan["positions"].long()
    ref = torch.where((p < 150)[..., None], rows[p.clamp(max=149)].double(), 0.0).sum(1)
    assert_within(y, ref, ref.abs() * 4 * U32 + 4 * U32, "y")
    assert dispatch(normal((100, 64), 52), short).shape == (150, 64)


def test_autograd():
    """A mixture with plain products between, against the same in float64."""
    from lm_head_linear_chunked_gb300.expert_rows import combine, dispatch, expert_plan
    T, k, E, H = 200, 2, 5, 96
    x, up = normal((4, 50, H), 60).requires_grad_(True), normal((E, H, H), 61, std=H ** -0.5).requires_grad_(True)
    w = normal((4, 50, k), 62).requires_grad_(True)
    experts = experts_of(T, k, E, 63, "unused").view(4, 50, k)
    mask = normal((4, 50), 64) > -1
    c = normal((4, 50, H), 65)
    plan = expert_plan(experts, E, mask, 8)
    rows = dispatch(x, plan)
    ends = plan["offsets"].tolist()
    out = torch.cat([rows[a:b] @ up[e] for e, (a, b) in enumerate(zip(ends, ends[1:]))] + [rows[ends[-1]:] @ up[0]])
    got = torch.autograd.grad((combine(out, w, plan) * c).sum(), (x, up, w))
    xd, ud, wd = (t.detach().double().requires_grad_(True) for t in (x, up, w))
    every = torch.einsum("abh,ehf->abef", xd, ud)
    on = ((experts >= 0) & mask[..., None])
    picked = every.gather(2, experts.clamp(min=0)[..., None].expand(*experts.shape, H)) * (wd * on)[..., None]
    want = torch.autograd.grad((picked.sum(2) * c.double()).sum(), (xd, ud, wd))
    torch.backends.cuda.matmul.allow_tf32 = False
    for g, r, terms in zip(got, want, (H * k, 2 * T, H)):
        assert (g.double() - r).abs().max() <= 4 * terms * U32 * r.abs().max() * 8  # products and sums of `terms` in FP32
    assert not dispatch(x.detach(), plan).requires_grad


@pytest.mark.parametrize("H", [8, 65, 66, 128, 256, 264, 1601, 8200])
@pytest.mark.parametrize("k", [1, 2, 3, 8, 11])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_unused_slots_beside_a_gradient_that_is_not_finite(H, k, dtype):
    """A slot without a row has the weight's gradient 0, whatever dy and the token's other slots hold."""
    from lm_head_linear_chunked_gb300.expert_rows import combine_backward, expert_plan
    T, E = 30, 16
    t, j = torch.arange(T, device="cuda")[:, None], torch.arange(k, device="cuda")
    experts = torch.where((t + j * j) % 3 == 0, -1, (t + j) % E)
    mask = t[:, 0] % 7 != 5
    plan = expert_plan(experts, E, mask, 4)
    dy, rows = normal((T, H), 70, DTYPES[dtype]), normal((plan["slots"].shape[0], H), 71, DTYPES[dtype])
    for i, v in enumerate((float("inf"), float("-inf"), float("nan"))):
        dy[i::5, (7 * i) % H] = v
    rows[plan["slots"] < 0] = float("nan")
    p = plan["positions"].long()
    has = p >= 0
    assert torch.equal(has, (experts >= 0) & mask[:, None])
    each = rows[p.clamp(min=0)].double() * dy.double()[:, None]
    ref = torch.where(has, each.sum(2), 0.0)
    for wtype in (torch.float32, DTYPES[dtype]):
        got = combine_backward(dy, rows, normal((T, k), 72, wtype), plan)
        assert not got["grad_weights"][~has].any()
        assert torch.equal(got["grad_weights"].isnan(), ref.isnan()) and torch.equal(got["grad_weights"].isinf(), ref.isinf())
        finite = has & ref.isfinite()
        tol = each.abs().sum(2)[finite] * (sum_depth(H) + H / 32 + 4) * U32 + ref[finite].abs() * half_step(wtype) + tiny(wtype)
        assert_within(got["grad_weights"][finite], ref[finite], tol, "grad_weights")
        assert not got["grad_rows"][plan["slots"] < 0].any()
