"""The balance loss (balance_loss.py) on the GPU against its formulas in
float64.  The counts are whole numbers and have to be equal.

Tolerances: with a = max|z| of a group, the exponent's argument is off by at
most (4 a + 16) 2^-24, which is the relative error of one exponential; p has
that twice, and its row sum adds at most E/32 + 16 terms in sequence:
  e_p = (8 a + 64 + E/32) 2^-24, relative.
The mean over tokens adds at most T terms in sequence.  The gradient
p (f' - sum f' p), f' = f - 1, has e_p of the sum of its terms' magnitudes
three times over, and one rounding to its type."""
import pytest
import torch

import lm_head_linear_chunked_gb300 as lce
from tests.op_util import DTYPES, U32, assert_within, half_step, normal, tiny

pytestmark = pytest.mark.gpu


def problem(G, T, E, k, dtype, seed, masked=False, index=torch.int64, lean=0.8):
    z = (normal((G, T, E), seed) + normal((G, 1, E), seed + 1, std=lean)).to(DTYPES[dtype])
    experts = z.float().topk(k, dim=-1).indices.to(index)
    mask = normal((T,), seed + 2) > -0.8 if masked else None
    return z, experts, mask


def formulas(z, experts, mask, scale=1.0, reduction="mean"):
    G, T, E = z.shape
    k = experts.shape[-1]
    keep = torch.ones((G, T), dtype=torch.bool, device=z.device) if mask is None else mask.expand(G, T)
    out = {"group_loss": [], "counts": [], "n_valid": [], "grad": [], "size": []}
    for g in range(G):
        zz = torch.where(keep[g, :, None], z[g].double(), 0.0)
        p = torch.softmax(zz, 1)
        e = experts[g][keep[g]].reshape(-1).long()
        c = torch.bincount(e[e >= 0], minlength=E)
        n = int(keep[g].sum())
        f = c.double() * E / (k * max(n, 1))
        out["counts"].append(c)
        out["n_valid"].append(n)
        out["group_loss"].append((f * (p * keep[g, :, None]).sum(0) / max(n, 1)).sum())
        s = scale / max(n, 1) / (G if reduction == "mean" else 1)
        fc = f - 1
        d = s * p * (f - (p @ f)[:, None]) * keep[g, :, None]
        size = abs(s) * p * (fc.abs() + (p @ fc.abs())[:, None])
        out["grad"].append(d)
        out["size"].append(size)
    r = {k: torch.stack(v) if torch.is_tensor(v[0]) else torch.tensor(v, device=z.device) for k, v in out.items()}
    r["loss"] = r["group_loss"].mean() if reduction == "mean" else r["group_loss"].sum()
    return r


def check(z, experts, mask, got, scale=1.0, reduction="mean"):
    r = formulas(z, experts, mask, scale, reduction)
    G, T, E = z.shape
    kept = z if mask is None else z[mask.expand(G, T)]
    a = float(kept.abs().masked_fill(kept.abs() == float("inf"), 0).max()) if kept.numel() else 0.0
    e_p = (8 * a + 64 + E / 32) * U32
    if "loss" in got:
        assert torch.equal(got["counts"].reshape(G, E), r["counts"])
        assert torch.equal(got["n_valid"], r["n_valid"])
        e = e_p + (T + 16) * U32
        assert_within(got["group_loss"], r["group_loss"], e * r["group_loss"].abs(), "group_loss")
        assert_within(got["loss"].reshape(()), r["loss"], e * r["group_loss"].abs().sum() / (
            G if reduction == "mean" else 1) + U32 * r["loss"].abs(), "loss")
        assert lce.lce_check_status(got["ws"], torch.cuda.current_stream()) == 0
    if "grad_logits" in got:
        t = z.dtype
        assert got["grad_logits"].dtype == t
        u = half_step(t)
        assert_within(got["grad_logits"].reshape(z.shape), r["grad"],
                      u * r["grad"].abs() + (1 + u) * (3 * e_p + 8 * U32) * r["size"] + tiny(t), "grad_logits")


def run(z, experts, mask, scale=1.0, reduction="mean"):
    from lm_head_linear_chunked_gb300.balance_loss import balance_backward, balance_forward, balance_fused
    g = torch.full((1,), scale, device="cuda")
    f = balance_forward(z, experts, mask, reduction)
    b = balance_backward(z, f["counts"], f["n_valid"], experts.shape[-1], mask, 1.0, g, reduction)
    check(z, experts, mask, {**f, **b}, scale, reduction)
    u = balance_fused(z, experts, mask, 1.0, g, reduction)
    check(z, experts, mask, u, scale, reduction)
    assert torch.equal(u["counts"], f["counts"])
    return f, b, u


@pytest.mark.parametrize("G,T,E,k", [(1, 1, 1, 1), (1, 1, 8, 2), (1, 509, 8, 2), (3, 130, 60, 4), (2, 33, 64, 6),
                                     (4, 1000, 128, 8), (1, 4099, 61, 4), (2, 257, 160, 6), (5, 64, 256, 8),
                                     (1, 300, 384, 8), (1, 77, 1024, 16), (40, 3, 16, 1), (1, 20001, 7, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_sizes(G, T, E, k, dtype):
    z, experts, mask = problem(G, T, E, k, dtype, G + T + E, masked=T % 2 == 1 and T > 1)
    run(z, experts, mask, scale=512.0)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_index_types_and_reductions(index, reduction):
    z, experts, mask = problem(3, 200, 64, 4, "bf16", 7, True, index)
    run(z, experts, mask, 0.25, reduction)


def test_unused_slots_are_not_counted():
    z, experts, mask = problem(2, 300, 16, 4, "fp32", 11, True)
    experts[normal(experts.shape, 12) > 1.0] = -1
    run(z, experts, mask)


def test_strided_logits():
    wide = normal((2, 90, 3, 40), 13, torch.bfloat16)
    for z in (wide[:, :, 1], wide[:, ::2, 0, :33], wide.transpose(0, 1)[:2, :, 2]):
        experts = z.float().topk(3, dim=-1).indices
        run(z, experts, None)
    z = wide[0, :, 0].T  # experts not contiguous: copied
    run(z[None], z[None].float().topk(2, dim=-1).indices, None)


def test_masks():
    """A mask of its own per group, a group left empty, and all of them empty."""
    z, experts, _ = problem(4, 150, 32, 2, "fp32", 17)
    mask = normal((4, 150), 18) > 0
    mask[2] = False
    run(z, experts, mask)
    f, b, u = run(z, experts, torch.zeros_like(mask))
    assert float(f["loss"]) == 0.0 and not b["grad_logits"].any() and not u["grad_logits"].any()


def test_masked_tokens_have_no_influence():
    z, experts, mask = problem(2, 333, 24, 3, "bf16", 19, True)
    ref = run(z, experts, mask)
    z2, e2 = z.clone(), experts.clone()
    z2[:, ~mask] = float("nan")
    z2[:, (~mask).nonzero()[0]] = float("inf")
    e2[:, ~mask] = 12345
    from lm_head_linear_chunked_gb300.balance_loss import balance_backward, balance_forward, balance_fused
    f = balance_forward(z2, e2, mask)
    u = balance_fused(z2, e2, mask)
    b = balance_backward(z2, f["counts"], f["n_valid"], 3, mask)
    for k in ("loss", "counts", "n_valid", "group_loss"):
        assert torch.equal(f[k], ref[0][k]) and torch.equal(u[k], ref[2][k])
    assert torch.equal(b["grad_logits"], ref[1]["grad_logits"]) and torch.equal(u["grad_logits"], ref[2]["grad_logits"])


def test_switched_off_experts():
    """Logits of minus infinity: p = 0 and no gradient there."""
    z, experts, mask = problem(1, 100, 32, 4, "fp32", 23)
    z[:, :, 20:] = -float("inf")
    experts = z.topk(4, dim=-1).indices
    f, b, u = run(z, experts, mask)
    assert not b["grad_logits"][:, :, 20:].any()


def test_an_even_load_costs_one():
    T, E = 512, 16
    z = torch.zeros((1, T, E), device="cuda")
    experts = (torch.arange(T, device="cuda") % E)[None, :, None]
    f, b, u = run(z, experts, None)
    assert float(f["loss"]) == 1.0 and not b["grad_logits"].any()


@pytest.mark.parametrize("bad", [16, -2, 1 << 40])
def test_an_index_out_of_range_is_reported(bad):
    from lm_head_linear_chunked_gb300.balance_loss import balance_forward, balance_loss
    z, experts, _ = problem(2, 50, 16, 2, "fp32", 29)
    experts[1, 7, 1] = bad
    f = balance_forward(z, experts)
    assert lce.lce_check_status(f["ws"], torch.cuda.current_stream()) == 8 and torch.isnan(f["loss"]).all()
    with pytest.raises(lce.LCEError) as e:
        balance_loss(z, experts, check=True)
    assert e.value.status == 8


def test_autograd_and_differences():
    from lm_head_linear_chunked_gb300.balance_loss import balance_loss
    z, experts, mask = problem(2, 64, 12, 2, "fp32", 31, True)
    z.requires_grad_(True)
    loss, counts = balance_loss(z, experts, mask, check=True)
    (loss * 3.0).backward()
    check(z.detach(), experts, mask, {"grad_logits": z.grad}, 3.0)
    assert not counts.requires_grad and loss.shape == ()
    # central differences: the third derivative of the loss along a unit direction is at most of order the
    # largest f times a few; the loss has fp32 rounding of its tokens' sums
    with torch.no_grad():
        v = normal(z.shape, 32)
        v /= v.norm()
        h = 2.0 ** -3
        f = [float(balance_loss(z + s * v, experts, mask)[0].double()) for s in (h, -h)]
        want = float((z.grad.double() * v).sum()) / 3.0
        top = float(counts.double().max()) * 12 / (2 * int(mask.sum()))
        assert abs((f[0] - f[1]) / (2 * h) - want) <= top * (h * h / 64 + 64 * U32 / h)


def test_two_dimensional_logits_and_no_grad():
    from lm_head_linear_chunked_gb300.balance_loss import balance_loss
    z, experts, mask = problem(1, 90, 20, 3, "bf16", 37, True)
    loss, counts = balance_loss(z[0], experts[0], mask)
    loss3, counts3 = balance_loss(z, experts, mask)
    assert counts.shape == (20,) and torch.equal(counts, counts3[0]) and torch.equal(loss, loss3)


def test_side_stream_repeats_and_graph_capture():
    from lm_head_linear_chunked_gb300.balance_loss import balance_fused
    z, experts, mask = problem(3, 700, 64, 4, "bf16", 41, True)
    ref = balance_fused(z, experts, mask)
    names = ("loss", "group_loss", "counts", "n_valid", "grad_logits")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = balance_fused(z, experts, mask)
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], ref[k]) for k in names)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = balance_fused(z, experts, mask)
    for _ in range(2):
        for k in names:
            out[k].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], ref[k]) for k in names)


@pytest.mark.parametrize("E", [7, 60, 64, 128, 200, 1024])  # single elements, 8- and 16-byte vectors, one and several a lane
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_of_large_logits(E, dtype):
    """Rows of one large value have the softmax of a row of zeros, 1 / E, exactly as that row does (the largest is
    subtracted first, so nothing is rounded); a row with one expert far above the rest has 1 and 0."""
    t = DTYPES[dtype]
    small, experts, _ = problem(1, 300, E, 2, dtype, 43)
    large = small.clone()
    low, high = torch.finfo(t).min, torch.finfo(t).max
    for i, v in enumerate((low, high, -1e30, 1e30, -1e10, 1e10, 3e9, -2.0 ** 40)):
        small[0, 7 * i] = 0
        large[0, 7 * i] = v
    # e^-x is 0 in 64 bits for x > 745, so the small row stands for all of these
    for i, (rest, one) in enumerate(((low, 0.0), (low, high), (-1e10, 1e10), (-1e10, -1e9), (1e9, 1e10))):
        small[0, 100 + i], large[0, 100 + i] = -1000, rest
        small[0, 100 + i, E // 2], large[0, 100 + i, E // 2] = 0, one
    from lm_head_linear_chunked_gb300.balance_loss import balance_backward, balance_forward, balance_fused
    f = balance_forward(large, experts)
    b = balance_backward(large, f["counts"], f["n_valid"], 2)
    plain = small.clone()
    plain[0, 100:105] = plain[0, 100:105].clamp(min=-16)  # only for the size of the tolerance
    a = float(plain.abs().max())
    for got in ({**f, **b}, balance_fused(large, experts)):
        for k in ("loss", "group_loss", "grad_logits"):
            assert not torch.isnan(got[k]).any(), k
        r = formulas(small, experts, None)
        e_p = (8 * a + 64 + E / 32) * U32
        e = e_p + (300 + 16) * U32
        assert_within(got["loss"].reshape(()), r["loss"], (e + U32) * r["loss"].abs(), "loss")
        u = half_step(t)
        assert_within(got["grad_logits"].reshape(small.shape), r["grad"],
                      u * r["grad"].abs() + (1 + u) * (3 * e_p + 8 * U32) * r["size"] + tiny(t), "grad_logits")


@pytest.mark.parametrize("kind", ["unused slots", "unlikely experts"])
def test_losses_far_below_one(kind):
    """The loss is 1 + sum_e (f_e - 1) P_e, whose terms add up to at most 1 + loss in size."""
    z, experts, mask = problem(3, 257, 16, 2, "fp32", 47, True)
    if kind == "unused slots":
        experts[normal(experts.shape, 48) > -2.5] = -1
    else:
        z[:, :, 0] += 15
        experts[:] = 1 + experts % 15
    r = formulas(z, experts, mask)
    assert 0 <= float(r["group_loss"].max()) < 0.05
    a = float(z[:, mask].abs().max())
    e = (8 * a + 64 + 16 / 32 + 257 + 16) * U32
    from lm_head_linear_chunked_gb300.balance_loss import balance_fused
    f = balance_fused(z, experts, mask)
    assert_within(f["group_loss"], r["group_loss"], e * (1 + r["group_loss"]), "group_loss")
    assert_within(f["loss"].reshape(()), r["loss"], (e + U32) * (1 + r["loss"]), "loss")
