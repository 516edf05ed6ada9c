"""RMS norm on the GPU against float64."""
import pytest
import torch

from tests.op_util import DTYPES, U32, assert_within, half_step, normal, tiny
from tests.row_refs import rms_backward_ref, rms_ref, rms_tolerance, sum_depth

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 7), (5, 64), (4, 128), (7, 200), (33, 1000), (2, 1601), (9, 1024), (130, 1024), (17, 2560), (6, 4096),
          (700, 4096), (3, 8192), (5, 8200), (2, 16384), (2, 16400), (3, 40001), (1000, 72), (611, 2049)]
EPS = 1e-5


def inputs(rows, H, dtype, wtype, seed=0):
    t, w = DTYPES[dtype], DTYPES[wtype]
    return (normal((rows, H), seed + 1, t, 1.5, 0.2), normal((rows, H), seed + 2, t, 2.0),
            normal((H,), seed + 3, w, 0.2, 1.0), normal((rows, H), seed + 4, t, 0.5), normal((rows, H), seed + 5, t, 0.5))


def check_backward(dy, s, w, rstd, ds, got, wtype):
    """Against the formula, term by term: the mean over the row is off by the depth of its sum times the mean of the
    magnitudes; products and differences by half a step each; the column sums by at most the rows (any order)."""
    rows, H = s.shape
    dx, dw = rms_backward_ref(dy, s, w, rstd, ds)
    t, r = s.dtype, rstd.double()[:, None]
    xh = s.double() * r
    g = dy.double() * (1 if w is None else w.double())
    m = (g * xh).abs().mean(1, keepdim=True)
    tol = r * U32 * (5 * g.abs() + (sum_depth(H) + 8) * xh.abs() * m) + 2 * U32 * (0 if ds is None else ds.double().abs())
    assert_within(got["grad_x"], dx, tol + dx.abs() * half_step(t) + tiny(t), "grad_x")
    if w is not None:
        each = (dy.double() * xh).abs().sum(0)
        assert_within(got["grad_weight"], dw, each * (rows + 4) * U32 + dw.abs() * half_step(wtype) + tiny(wtype), "grad_weight")


@pytest.mark.parametrize("rows,H", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_forward_and_backward(rows, H, dtype, wtype):
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_backward, rms_norm_forward
    x, res, w, dy, ds = inputs(rows, H, dtype, wtype)
    for residual, weight in ((None, w), (res, w), (res, None)):
        f = rms_norm_forward(x, weight, residual, EPS)
        s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
        assert torch.equal(f["sum"], s)
        y, rstd = rms_ref(s, weight, EPS)
        assert_within(f["y"], y, rms_tolerance(y, H, x.dtype), "y")
        assert_within(f["rstd"], rstd, rstd * (sum_depth(H) / 2 + 6) * U32, "rstd")
        check_backward(dy, s, weight, f["rstd"], ds if residual is not None else None,
                       rms_norm_backward(dy, s, weight, f["rstd"], ds if residual is not None else None), w.dtype)


@pytest.mark.parametrize("rows,H", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("group", [0, 128])
def test_fp8(rows, H, dtype, wtype, group):
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_fp8
    x, res, w, _, _ = inputs(rows, H, dtype, wtype, 10)
    for residual in (None, res):
        f = rms_norm_fp8(x, w, residual, EPS, group)
        s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
        assert torch.equal(f["sum"], s)
        y, _ = rms_ref(s, w, EPS)
        width = group or H
        wide = torch.nn.functional.pad(y, (0, -H % width)).view(rows, -1, width)
        scales = wide.abs().amax(2).clamp(min=2.0 ** -100) / 448
        near = (sum_depth(H) / 2 + 10) * U32  # y as above, then the largest, the division and the product
        assert_within(f["scales"], scales, scales * near, "scales")
        assert f["q"].dtype == torch.float8_e4m3fn and f["q"].shape == x.shape
        # against the kernel's own scales: e4m3 steps are 2^-3 of the value, 2^-9 below 2^-6
        got = f["scales"].double()[:, :, None]
        q = (wide / got).view(rows, -1)[:, :H]
        assert_within(f["q"].float(), q, q.abs() * (2.0 ** -4 + near) + 2.0 ** -10, "q")


def test_rows_that_are_zero_tiny_or_not_finite():
    """Each row for itself: what one holds does not reach another."""
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_forward, rms_norm_fp8
    for H in (96, 1024, 4096, 1601, 20000):
        x = normal((8, H), 20)
        x[1] = 0.0
        x[2] = x[2] * 1e-30  # squares below FP32's range: eps decides
        x[3, H // 2] = float("inf")
        x[4, H // 3] = float("nan")
        x[5, -1] = -float("inf")
        x[6] = x[6] * 1e16   # their sum is near FP32's range
        w = normal((H,), 21, mean=1.0, std=0.1)
        f = rms_norm_forward(x, w, None, EPS)
        y, _ = rms_ref(x, w, EPS)
        fine = torch.tensor([0, 1, 2, 6, 7], device="cuda")
        assert_within(f["y"][fine], y[fine], rms_tolerance(y[fine], H, x.dtype), "y")
        assert torch.equal(f["y"].isnan(), y.isnan())
        for group in (0, 128):
            e = rms_norm_fp8(x, w, None, EPS, group)
            q, scales = e["q"].float(), e["scales"]
            assert bool(q[fine].isfinite().all()) and bool(scales[fine].isfinite().all())
            assert not q[1].any() and bool((scales[1] == 2.0 ** -100 / 448).all())
            at = lambda c: c // group if group else 0  # noqa: E731
            for r, c in ((3, H // 2), (4, H // 3), (5, H - 1)):
                assert bool(scales[r, at(c)].isnan()) and bool(q[r, c].isnan())
            assert bool(scales[4].isnan().all())  # rstd is NaN
            assert int(scales[3].isnan().sum()) == 1
        assert bool(torch.isfinite(rms_norm_forward(x[:3].bfloat16(), None, None, 0.0)["y"][0]).all())


@pytest.mark.parametrize("H", [64, 72, 1024, 2560, 4096, 1601, 8200, 20001])
def test_strides_and_alignment(H):
    """Rows further apart than their width, bases off every vector's boundary, more dimensions, broadcast residuals."""
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm, rms_norm_backward, rms_norm_forward, rms_norm_fp8
    wide = normal((6, H + 24), 30, torch.bfloat16)
    w = normal((H + 1,), 31, torch.bfloat16, 0.1, 1.0)
    for cut in (slice(8, 8 + H), slice(0, H), slice(1, 1 + H), slice(2, 2 + H)):
        for weight in (w[:H], w[1:]):
            x, r = wide[:3, cut], wide[3:, cut]
            want = rms_norm_forward(x.contiguous(), weight.clone(), r.contiguous(), EPS)
            got = rms_norm_forward(x, weight, r, EPS)
            ref, _ = rms_ref(want["sum"], weight, EPS)
            assert torch.equal(got["sum"], want["sum"])
            assert_within(got["y"], ref, rms_tolerance(ref, H, x.dtype), "y")
            b = rms_norm_backward(x, r, weight, want["rstd"], x)
            check_backward(x, r, weight, want["rstd"], x, b, weight.dtype)
            q = rms_norm_fp8(x, weight, r, EPS)
            assert torch.equal(q["sum"], want["sum"])
            deq = torch.nn.functional.pad(q["q"].float(), (0, -H % 128)).view(3, -1, 128) * q["scales"][:, :, None]
            deq = deq.view(3, -1)[:, :H].double()
            most = q["scales"].double().repeat_interleave(128, 1)[:, :H]
            assert_within(deq, ref, ref.abs() * (2.0 ** -4 + 64 * U32) + most * 2.0 ** -10, "dequantized")
    x4 = normal((2, 3, 4, H), 32)
    y, s = rms_norm(x4, None, x4[:1].expand(2, 3, 4, H), EPS)
    ref, _ = rms_ref(x4 + x4[:1], None, EPS)
    assert y.shape == s.shape == x4.shape
    assert_within(y, ref, rms_tolerance(ref, H, y.dtype), "y")
    assert torch.equal(rms_norm(torch._neg_view(x4), None, None, EPS), rms_norm(-x4, None, None, EPS))


@pytest.mark.parametrize("dtype,H", [("fp32", H) for H in (255, 4095, 4097, 6399, 6401, 8188, 8191, 8192)] +
                         [(d, H) for d in ("bf16", "fp16") for H in (255, 510, 4095, 4097, 8190, 8191, 8192, 16376, 16384)])
def test_every_form_at_its_widest(dtype, H):
    """With a residual and the sum's gradient, which take the most shared memory."""
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_backward, rms_norm_forward, rms_norm_fp8
    for rows, wtype in ((3, dtype), (700, "fp32")):
        x, res, w, dy, ds = inputs(rows, H, dtype, wtype, 50)
        f = rms_norm_forward(x, w, res, EPS)
        ref, _ = rms_ref(f["sum"], w, EPS)
        assert torch.equal(f["sum"], x + res)
        assert_within(f["y"], ref, rms_tolerance(ref, H, x.dtype), "y")
        check_backward(dy, f["sum"], w, f["rstd"], ds, rms_norm_backward(dy, f["sum"], w, f["rstd"], ds), w.dtype)
        check_backward(dy, f["sum"], w, f["rstd"], None, rms_norm_backward(dy, f["sum"], w, f["rstd"]), w.dtype)
        assert torch.equal(rms_norm_fp8(x, w, res, EPS)["sum"], f["sum"])


def test_negated_views():
    """Memory that stands for other values, in every place that takes a tensor."""
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_backward, rms_norm_forward, rms_norm_fp8
    x, r, d, s = (normal((5, 320), k) for k in (34, 35, 36, 37))
    w = normal((320,), 38)
    neg = torch._neg_view
    want, got = rms_norm_forward(-x, -w, -r, EPS), rms_norm_forward(neg(x), neg(w), neg(r), EPS)
    assert all(torch.equal(want[k], got[k]) for k in want)
    want, got = rms_norm_fp8(-x, -w, -r, EPS), rms_norm_fp8(neg(x), neg(w), neg(r), EPS)
    assert all(torch.equal(want[k].float(), got[k].float()) for k in want)
    rstd = rms_norm_forward(-x, None, None, EPS)["rstd"]
    want, got = rms_norm_backward(-d, -x, -w, rstd, -s), rms_norm_backward(neg(d), neg(x), neg(w), rstd, neg(s))
    assert all(torch.equal(want[k], got[k]) for k in want)
    with pytest.raises(TypeError):
        rms_norm_backward(d, x, w, neg(rstd), s)


def test_autograd():
    """Through the module: y and the sum used, one of them, and neither's gradient asked for."""
    from lm_head_linear_chunked_gb300.rms_norm import RMSNorm, rms_norm, rms_norm_backward, rms_norm_forward
    m = RMSNorm(256, EPS, device="cuda", dtype=torch.bfloat16)
    with torch.no_grad():
        m.weight += normal((256,), 40, torch.bfloat16, 0.1)
    x, r = (normal((2, 5, 256), k, torch.bfloat16).requires_grad_(True) for k in (41, 42))
    cy, cs = (normal((2, 5, 256), k, torch.bfloat16) for k in (43, 44))
    f = rms_norm_forward(x.detach(), m.weight.detach(), r.detach(), EPS)
    leaves = (x, r, m.weight)

    def want(dy, ds):
        return rms_norm_backward(dy, f["sum"], m.weight.detach(), f["rstd"], ds)

    y, s = m(x, r)
    both = torch.autograd.grad((y, s), leaves, (cy, cs))
    d = want(cy, cs)
    assert torch.equal(both[0], d["grad_x"]) and torch.equal(both[1], d["grad_x"]) and torch.equal(both[2], d["grad_weight"])
    y, s = m(x, r)
    only_y = torch.autograd.grad(y, leaves, cy)
    d = want(cy, None)
    assert torch.equal(only_y[0], d["grad_x"]) and torch.equal(only_y[2], d["grad_weight"])
    y, s = m(x, r)
    only_s = torch.autograd.grad(s, (x, r), cs)
    assert torch.equal(only_s[0], cs) and torch.equal(only_s[1], cs)
    y = m(x)
    alone = torch.autograd.grad(y, (x,), cy)[0]
    f1 = rms_norm_forward(x.detach(), m.weight.detach(), None, EPS)
    assert torch.equal(alone, rms_norm_backward(cy, x.detach(), m.weight.detach(), f1["rstd"])["grad_x"])
    assert not rms_norm(x.detach(), m.weight.detach()).requires_grad
    y, s = m(x, r)  # gradients that arrive expanded, and leaves that meet twice
    (y.sum() + s.sum() + m(x, x)[0].sum()).backward()
    assert x.grad.shape == x.shape and bool(x.grad.isfinite().all())


def test_no_rows():
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_backward, rms_norm_forward, rms_norm_fp8
    x, w = torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda")
    f = rms_norm_forward(x, w, x)
    assert f["y"].shape == (0, 64) and f["rstd"].shape == (0,)
    assert rms_norm_fp8(x, w)["scales"].shape == (0, 1)
    assert not rms_norm_backward(x, x, w, f["rstd"])["grad_weight"].any()


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 31, 33, 1000, 40001])
@pytest.mark.parametrize("H,dtype", [(8, "bf16"), (24, "bf16"), (64, "fp16"), (72, "bf16"), (128, "fp16"), (136, "bf16"), (32, "fp32"),
                                     (48, "fp32"), (64, "fp32"), (68, "fp32"), (82, "bf16"), (87, "bf16"), (87, "fp32"), (130, "fp16"),
                                     (201, "fp32"), (250, "bf16"), (255, "fp16"), (258, "bf16"), (500, "fp16"), (576, "bf16"),
                                     (704, "fp16"), (776, "bf16")])
def test_narrow_rows(rows, H, dtype):
    """Several rows to a warp: rows that end inside one, and rows beside one that is not finite."""
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_backward, rms_norm_forward, rms_norm_fp8
    x, res, w, dy, ds = inputs(rows, H, dtype, dtype, 70)
    f = rms_norm_forward(x, w, res, EPS)
    y, rstd = rms_ref(f["sum"], w, EPS)
    assert_within(f["y"], y, rms_tolerance(y, H, x.dtype), "y")
    assert_within(f["rstd"], rstd, rstd * (sum_depth(H) / 2 + 6) * U32, "rstd")
    check_backward(dy, f["sum"], w, f["rstd"], ds, rms_norm_backward(dy, f["sum"], w, f["rstd"], ds), w.dtype)
    for group in (0, 128):
        q = rms_norm_fp8(x, w, res, EPS, group)
        scale = q["scales"].repeat_interleave(group or H, 1)[:, :H].double()
        assert_within(q["q"].double(), y / scale, (y / scale).abs() * (2.0 ** -4 + 64 * U32) + 2.0 ** -10, "q")
    bad = x.clone()
    bad[rows // 2, H // 2] = float("nan")
    g = rms_norm_forward(bad, w, res, EPS)
    fine = torch.arange(rows, device="cuda") != rows // 2
    assert torch.equal(g["y"][fine], f["y"][fine]) and bool(g["y"][~fine].isnan().all())
    d = rms_norm_backward(dy, g["sum"], w, g["rstd"], ds)
    assert bool(d["grad_x"][fine].isfinite().all()) and bool(d["grad_weight"].isnan().all())
    # its gradient zero: the row adds nothing that is not NaN itself, and the other columns' sums are those of the others
    zero = rms_norm_backward(torch.where(fine[:, None], dy, 0), torch.where(fine[:, None], f["sum"], 0), w, f["rstd"])["grad_weight"]
    part = rms_norm_backward(dy[fine], f["sum"][fine], w, f["rstd"][fine])["grad_weight"]
    each = (dy.double() * f["sum"].double() * f["rstd"].double()[:, None]).abs().sum(0)
    assert_within(zero, part.double(), each * 2 * (rows + 4) * U32 + 3 * half_step(w.dtype) * part.double().abs() + 3 * tiny(w.dtype), "sums")


@pytest.mark.parametrize("H", [64, 96, 250, 1024, 1601, 4096, 8192, 16384, 16400, 40001])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("group", [0, 128])
def test_8_bit_values_bit_by_bit(H, dtype, group):
    """q is rounded from y times the rounded reciprocal of the scale.  Even widths have a weight whose
    quotients by the scale lie between two values of e4m3; where rstd = 1 dividing would round some the other way."""
    from lm_head_linear_chunked_gb300.rms_norm import rms_norm_forward, rms_norm_fp8
    t, rows = DTYPES[dtype], 5
    m = torch.arange(H, device="cuda") % 128 % 120
    between = ((8 + m % 8).float() * 2 + 1) / 16 * 2.0 ** (m // 8 - 7).float()
    between[torch.arange(H, device="cuda") % 128 == min(H, 128) - 1] = 448
    c = torch.randint(1 << 15, 1 << 16, (-(-H // 128),), generator=torch.Generator().manual_seed(6)).cuda() * 2.0 ** -15
    w = between * c.repeat_interleave(128)[:H]
    x = torch.where(normal((rows, H), 30) > 0, 1.0, -1.0).to(t)
    if H % 2:
        x, w = normal((rows, H), 31, t), normal((H,), 32)
    rstd = rms_norm_forward(x, w, None, 0.0)["rstd"].cpu()
    assert H & (H - 1) or bool((rstd == 1).all())
    got = rms_norm_fp8(x, w, None, 0.0, group)
    y = x.float().cpu() * rstd[:, None] * w.cpu()
    width = group or H
    wide = torch.nn.functional.pad(y, (0, -H % width)).view(rows, -1, width)
    scales = wide.abs().amax(2) / 448
    assert torch.equal(got["scales"].cpu(), scales)
    q = (wide * (1 / scales)[:, :, None]).view(rows, -1)[:, :H].to(torch.float8_e4m3fn)
    assert torch.equal(got["q"].cpu().view(torch.uint8), q.view(torch.uint8))
    if group and H & (H - 1) == 0 and H >= 1024:
        assert not torch.equal((wide / scales[:, :, None]).view(rows, -1)[:, :H].to(torch.float8_e4m3fn).view(torch.uint8), q.view(torch.uint8))
