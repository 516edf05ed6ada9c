"""Layer norm (layer_norm.py) on the GPU against its formulas in float64.

Tolerances, element by element, with u the half step of the output's type
and 2^-24 that of fp32.  The forward sums H values in an order that adds at
most H/32 + 16 terms one after the other, so mean and centred values are off
by at most (H/32 + 16) 2^-24 of the row's largest |x| (in units of 1/rstd:
A = rstd max|x|), and the remaining operations add a few roundings of what
they combine.  The backward's row sums are bounded in the same way by the
sums of magnitudes.  The column sums add at most `rows` terms in sequence."""
import pytest
import torch

from tests.op_util import DTYPES, U32, assert_within, half_step, normal, tiny

pytestmark = pytest.mark.gpu


def formulas(x, w, b, dy, eps):
    x, dy = x.double(), dy.double()
    H = x.shape[-1]
    w = torch.ones(H, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros(H, dtype=torch.float64, device=x.device) if b is None else b.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    rows = tuple(range(x.dim() - 1))
    return {"mean": mean, "rstd": rstd, "xh": xh, "y": xh * w + b, "w": w, "b": b, "g": g, "dx": dx,
            "dw": (dy * xh).sum(rows), "db": dy.sum(rows), "x": x, "dy": dy}


def check(x, w, b, dy, eps, got):
    r = formulas(x, w, b, dy, eps)
    H, rows = x.shape[-1], x.numel() // x.shape[-1]
    k = (H / 32 + 16) * U32
    A = r["rstd"] * r["x"].abs().amax(-1, keepdim=True)  # |x| in units of the row's deviation
    u = half_step(x.dtype)
    e_xh = k * (A + r["xh"].abs() * (2 + A))             # centring, then rstd's own error
    if "y" in got:
        assert_within(got["y"], r["y"], u * r["y"].abs() + (1 + u) * (e_xh * r["w"].abs() + 4 * U32 * (
            r["xh"].abs() * r["w"].abs() + r["b"].abs())) + tiny(x.dtype), "y")
    if got.get("mean") is not None:
        assert_within(got["mean"], r["mean"].reshape(-1), (k * r["x"].abs().amax(-1)).reshape(-1) + tiny(torch.float32),
                      "mean")
        assert_within(got["rstd"], r["rstd"].reshape(-1), (k * (2 + A) * r["rstd"]).reshape(-1), "rstd")
    g1 = r["g"].abs().mean(-1, keepdim=True)
    g2 = (r["g"] * r["xh"]).abs().mean(-1, keepdim=True)
    e_g2 = k * g2 + (r["g"].abs() * e_xh).mean(-1, keepdim=True)
    if got.get("grad_x") is not None:
        parts = r["g"].abs() + g1 + r["xh"].abs() * g2
        e = r["rstd"] * (k * (parts + g1) + e_xh * g2 + r["xh"].abs() * e_g2 + parts * k * (2 + A))
        assert_within(got["grad_x"], r["dx"], u * r["dx"].abs() + (1 + u) * e + tiny(x.dtype), "grad_x")
    dims = tuple(range(x.dim() - 1))
    for name, ref, size, term in (("grad_weight", "dw", (r["dy"] * r["xh"]).abs().sum(dims),
                                   (r["dy"].abs() * e_xh).sum(dims)),
                                  ("grad_bias", "db", r["dy"].abs().sum(dims), 0)):
        if got.get(name) is not None:
            v = half_step(got[name].dtype)
            assert_within(got[name], r[ref], v * r[ref].abs() + (1 + v) * ((rows + 16) * U32 * size + term)
                          + tiny(got[name].dtype), name)


def run(x, w, b, dy, eps=1e-5):
    from lm_head_linear_chunked_gb300.layer_norm import layer_norm_backward, layer_norm_forward
    f = layer_norm_forward(x, w, b, eps)
    d = layer_norm_backward(dy, x, w, f["mean"], f["rstd"], grad_dtype=None if b is None else b.dtype)
    return {**f, **d}


SHAPES = [(1, 1), (1, 7), (3, 64), (5, 1000), (2, 1601), (17, 4096), (700, 2560), (1025, 8), (2, 33000), (1, 70001),
          (4099, 129), (9, 16392), (33, 8192), (1300, 512), (64, 5120)]


@pytest.mark.parametrize("rows,H", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_forward_and_backward(rows, H, dtype, wtype):
    t, v = DTYPES[dtype], DTYPES[wtype]
    x = normal((rows, H), 1, t, std=1.5, mean=0.3)
    w, b = normal(H, 2, v, std=0.2, mean=1.0), normal(H, 3, v, std=0.2)
    dy = normal((rows, H), 4, t, std=0.7)
    check(x, w, b, dy, 1e-5, run(x, w, b, dy))


@pytest.mark.parametrize("rows,H", [(1, 256), (2000, 256), (650, 1024), (3000, 2048), (5, 2562), (9, 4098), (7, 6001),
                                    (3, 8191), (5, 8200), (2, 12288), (611, 16384), (3, 16390), (10, 4104)])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_every_form(rows, H, dtype, wtype):
    """Widths on both sides of each choice of kernel, and more rows than blocks."""
    t, v = DTYPES[dtype], DTYPES[wtype]
    x = normal((rows, H), 41, t, std=0.5, mean=-0.7)
    w, b = normal(H, 42, v, std=0.2, mean=1.0), normal(H, 43, v, std=0.2)
    dy = normal((rows, H), 44, t, std=0.7)
    check(x, w, b, dy, 1e-6, run(x, w, b, dy, 1e-6))


def test_weight_and_bias_at_every_alignment():
    """A float32 weight that starts between 32-byte, 16-byte and 4-byte boundaries."""
    x, dy = normal((33, 512), 45, torch.bfloat16), normal((33, 512), 46, torch.bfloat16)
    w, b = normal(530, 47), normal(530, 48)
    for k in (0, 1, 2, 4, 8, 12):
        check(x, w[k:k + 512], b[k:k + 512], dy, 1e-5, run(x, w[k:k + 512], b[k:k + 512], dy))


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_without_weight_or_bias(weight, bias):
    x, dy = normal((37, 320), 5, torch.bfloat16), normal((37, 320), 6, torch.bfloat16)
    w = normal(320, 7, torch.float32) if weight else None
    b = normal(320, 8, torch.float32) if bias else None
    check(x, w, b, dy, 1e-5, run(x, w, b, dy))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("start,width", [(0, 256), (1, 256), (8, 264), (3, 251)])
def test_rows_of_a_wider_tensor(dtype, start, width):
    """Rows with a stride, at starts that break the 16-byte alignment."""
    t = DTYPES[dtype]
    x = normal((50, 1040), 9, t)[:, start:start + width]
    dy = normal((50, 777), 10, t)[:, start:start + width]
    w, b = normal(width + 1, 11, t)[1:], normal(width, 12, t)
    check(x, w, b, dy, 1e-5, run(x, w, b, dy))


def test_leading_dimensions_and_transposed_input():
    x = normal((6, 5, 192), 13, torch.bfloat16).transpose(0, 1)
    dy = normal((5, 6, 192), 14, torch.bfloat16)
    w, b = normal(192, 15, torch.bfloat16), normal(192, 16, torch.bfloat16)
    got = run(x, w, b, dy)
    assert got["y"].shape == x.shape and got["grad_x"].shape == x.shape
    check(x, w, b, dy, 1e-5, got)


@pytest.mark.parametrize("H", [64, 1000, 4096])
def test_rows_far_from_zero_and_constant_rows(H):
    """An offset of a thousand deviations, and rows whose variance is zero."""
    x = normal((6, H), 17, torch.float32, std=1.0, mean=1000.0)
    x[2] = 3.25
    x[4] = 0.0
    dy = normal((6, H), 18)
    w, b = normal(H, 19), normal(H, 20)
    got = run(x, w, b, dy)
    check(x, w, b, dy, 1e-5, got)
    assert torch.equal(got["y"][2], b) and torch.equal(got["y"][4], b)


@pytest.mark.parametrize("H", [96, 4096, 40000])
def test_a_bad_row_stays_by_itself(H):
    x, dy = normal((8, H), 21, torch.bfloat16), normal((8, H), 22, torch.bfloat16)
    w = normal(H, 23, torch.bfloat16)
    ref = run(x, w, None, dy)
    for bad in (float("inf"), float("nan")):
        z = x.clone()
        z[3, H // 2] = bad
        got = run(z, w, None, dy)
        keep = torch.arange(8, device="cuda") != 3
        assert torch.isnan(got["y"][3]).all() and torch.isnan(got["grad_x"][3]).all()
        for k in ("y", "grad_x"):
            assert torch.equal(got[k][keep], ref[k][keep])


@pytest.mark.parametrize("H", [8, 4096])
def test_no_rows(H):
    x = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    w, b = normal(H, 24, torch.bfloat16), normal(H, 25, torch.bfloat16)
    got = run(x, w, b, x)
    assert got["y"].shape == (0, H) and got["grad_x"].shape == (0, H)
    assert not got["grad_weight"].any() and not got["grad_bias"].any()


def test_gradients_alone():
    """Each gradient asked for by itself has the bits of the full call."""
    from lm_head_linear_chunked_gb300.layer_norm import layer_norm_backward
    x, dy, w = normal((130, 1024), 26, torch.bfloat16), normal((130, 1024), 27, torch.bfloat16), normal(1024, 28)
    full = run(x, w, None, dy)
    for names in (("grad_x",), ("grad_weight",), ("grad_bias",), ("grad_weight", "grad_bias"), ()):
        d = layer_norm_backward(dy, x, w, full["mean"], full["rstd"], "grad_x" in names, "grad_weight" in names,
                                "grad_bias" in names)
        for k in ("grad_x", "grad_weight", "grad_bias"):
            assert (d[k] is None) == (k not in names)
            assert d[k] is None or torch.equal(d[k], full[k])


def test_autograd_against_formula_and_differences():
    from lm_head_linear_chunked_gb300.layer_norm import LayerNorm
    torch.manual_seed(0)
    m = LayerNorm(96, device="cuda")
    with torch.no_grad():
        m.weight.copy_(normal(96, 29, mean=1.0, std=0.3))
        m.bias.copy_(normal(96, 30))
    x = normal((4, 3, 96), 31).requires_grad_(True)
    c = normal((4, 3, 96), 32)
    y = m(x)
    (y * c).sum().backward()
    check(x.detach(), m.weight.detach(), m.bias.detach(), c, 1e-5,
          {"y": y, "grad_x": x.grad, "grad_weight": m.weight.grad, "grad_bias": m.bias.grad})
    # central differences along a direction: h^2 / 6 of the third derivative (of order one
    # in these units) and fp32 rounding of about a thousand terms over 2 h
    h = 2.0 ** -7
    with torch.no_grad():
        for t, g in ((x, x.grad), (m.weight, m.weight.grad), (m.bias, m.bias.grad)):
            v = normal(t.shape, 33)
            v /= v.norm()
            keep = t.clone()
            f = []
            for s in (h, -h):
                t.copy_(keep + s * v)
                f.append((m(x).double() * c).sum())
            t.copy_(keep)
            slope = float((f[0] - f[1]) / (2 * h))
            want = float((g.double() * v).sum())
            size = float(c.norm() * m.weight.abs().max() + c.norm() * x.abs().max())
            assert abs(slope - want) <= size * (h * h + 64 * U32 / h)


def test_no_grad_gives_the_same_output_without_a_graph():
    from lm_head_linear_chunked_gb300.layer_norm import layer_norm
    x = normal((5, 256), 34, torch.bfloat16).requires_grad_(True)
    y = layer_norm(x)
    with torch.no_grad():
        z = layer_norm(x)
    assert y.requires_grad and not z.requires_grad and torch.equal(y, z)


def test_side_stream_repeats_and_graph_capture():
    x, dy = normal((515, 2560), 35, torch.bfloat16), normal((515, 2560), 36, torch.bfloat16)
    w, b = normal(2560, 37, torch.bfloat16), normal(2560, 38, torch.bfloat16)
    ref = run(x, w, b, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(x, w, b, dy)
    torch.cuda.current_stream().wait_stream(side)
    for k in ref:
        assert torch.equal(got[k], ref[k]), k
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = run(x, w, b, dy)
    for _ in range(2):
        for k in out:
            out[k].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k in ref:
            assert torch.equal(out[k], ref[k]), k
