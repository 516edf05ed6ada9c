"""The operators beside the head through the C ABI, with buffers that the
caller owns: the same bits as the torch front ends give, nothing written
outside the outputs and the workspace, no device memory taken by the calls,
every kernel seen by the profiling hook; and tensors of more than 2^32
bytes."""
import ctypes

import pytest
import torch

import lm_head_linear_chunked_gb300 as lce
from tests.op_util import normal

pytestmark = pytest.mark.gpu
GUARD = 512  # bytes of 0xA5 on both sides of a buffer


class Buffers:
    """Device buffers with guard bytes around them."""

    def __init__(self):
        self.all = []

    def take(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        size = n * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((GUARD + -(-size // 256) * 256 + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((raw, size))
        return raw[GUARD:GUARD + size].view(dtype).view(shape)

    def check(self):
        for raw, size in self.all:
            assert bool((raw[:GUARD] == 0xA5).all()) and bool((raw[GUARD + size:] == 0xA5).all())


def stream():
    return torch.cuda.current_stream()


@pytest.mark.parametrize("rows,H", [(5, 1), (300, 1601), (1000, 2560), (77, 512), (3, 40000)])
def test_layer_norm(rows, H):
    from lm_head_linear_chunked_gb300.layer_norm import layer_norm_backward, layer_norm_forward
    x, dy = normal((rows, H), 1, torch.bfloat16), normal((rows, H), 2, torch.bfloat16)
    w, b = normal(H, 3), normal(H, 4)
    B = Buffers()
    y, dx = B.take((rows, H), torch.bfloat16), B.take((rows, H), torch.bfloat16)
    mean, rstd, dw, db = (B.take((n,), torch.float32) for n in (rows, rows, H, H))
    nws = lce.lce_layer_norm_workspace_size(rows, H)
    ws = B.take((nws,), torch.uint8)
    lce.lce_layer_norm_forward(rows, H, lce.BF16, lce.F32, x, H, w, b, 1e-5, y, H, mean, rstd, stream())
    lce.lce_layer_norm_backward(rows, H, lce.BF16, lce.F32, dy, H, x, H, w, mean, rstd, dx, H, dw, db, ws, nws, stream())
    f = layer_norm_forward(x, w, b)
    d = layer_norm_backward(dy, x, w, f["mean"], f["rstd"])
    B.check()
    for got, want in ((y, f["y"]), (mean, f["mean"]), (rstd, f["rstd"]), (dx, d["grad_x"]), (dw, d["grad_weight"]),
                      (db, d["grad_bias"])):
        assert torch.equal(got, want)


@pytest.mark.parametrize("G,T,E,k", [(1, 40, 8, 2), (3, 700, 61, 4), (2, 5000, 128, 8)])
def test_balance_loss(G, T, E, k):
    from lm_head_linear_chunked_gb300.balance_loss import balance_backward, balance_fused
    z = normal((G, T, E), 5)
    experts = z.topk(k, dim=-1).indices
    mask = normal((T,), 6) > -1
    B = Buffers()
    loss, group = B.take((1,), torch.float32), B.take((G,), torch.float32)
    counts, n = B.take((G, E), torch.int64), B.take((G,), torch.int64)
    dz, dz2 = B.take((G, T, E), torch.float32), B.take((G, T, E), torch.float32)
    nws = lce.lce_balance_workspace_size(G, T, E, k)
    ws = B.take((nws,), torch.uint8)
    lce.lce_balance_fused(G, T, E, k, lce.F32, z, T * E, E, experts, 8, mask, 0, 2.0, None, loss, group, counts, n, dz, ws,
                          nws, stream(), 0)
    assert lce.lce_check_status(ws, stream()) == 0
    lce.lce_balance_backward(G, T, E, k, lce.F32, z, T * E, E, counts, n, mask, 0, 2.0, None, dz2, stream(), 0)
    B.check()
    f = balance_fused(z, experts, mask, grad_scale=2.0)
    for got, want in ((loss, f["loss"]), (group, f["group_loss"]), (counts, f["counts"]), (n, f["n_valid"]),
                      (dz, f["grad_logits"]),
                      (dz2, balance_backward(z, f["counts"], f["n_valid"], k, mask, 2.0)["grad_logits"])):
        assert torch.equal(got, want)
    # the forward alone
    lce.lce_balance_forward(G, T, E, k, lce.F32, z, T * E, E, experts.int(), 4, mask, 0, loss, None, counts, n, ws, nws,
                            stream(), 0)
    B.check()
    assert torch.equal(loss, f["loss"]) and torch.equal(counts, f["counts"])


@pytest.mark.parametrize("items,beams,V,n", [(1, 1, 1, 1), (2, 3, 5003, 6), (40, 16, 9000, 16), (1, 64, 2000, 64)])
def test_beams(items, beams, V, n):
    from lm_head_linear_chunked_gb300.beam import beam_reorder, beam_select
    z, s = normal((items, beams, V), 7, torch.float16), normal((items, beams), 8)
    over = normal((items, beams), 9) > 1.5
    B = Buffers()
    scores, tokens, parents = (B.take((items, n), t) for t in (torch.float32, torch.int64, torch.int64))
    ended = B.take((items, n), torch.bool)
    nws = lce.lce_beam_workspace_size(items, beams, V, n)
    ws = B.take((nws,), torch.uint8)
    lce.lce_beam_select(items, beams, V, n, lce.F16, z, V, s, over, 1, V // 2, scores, tokens, parents, ended, ws, nws,
                        stream())
    want = beam_select(z, s, n, over, 1, V // 2)
    for got, k in ((scores, "scores"), (tokens, "tokens"), (parents, "parents"), (ended, "finished")):
        assert torch.equal(got, want[k])
    state = normal((items * beams, 3, 10, 7), 10)
    out = B.take((items * n, 3, 4, 7), torch.float32)
    move = (lce.BeamState * 1)(lce.BeamState(state.data_ptr(), out.data_ptr(), 840, 336, 1, 0, 0, 3, 280, 112, 112))
    lce.lce_beam_reorder(items, beams, n, parents, move, 1, None, stream())
    B.check()
    assert torch.equal(out, beam_reorder([state[:, :, :4]], want["parents"])[0])


def test_no_device_memory_is_taken_and_every_kernel_is_seen():
    x = normal((4000, 1024), 11, torch.bfloat16)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    st = torch.empty((2, 4000), device="cuda")
    w = normal(1024, 12, torch.bfloat16)
    dw = torch.empty_like(w)
    nws = lce.lce_layer_norm_workspace_size(4000, 1024)
    ws = torch.empty(nws, dtype=torch.uint8, device="cuda")

    def calls():
        lce.lce_layer_norm_forward(4000, 1024, lce.BF16, lce.BF16, x, 1024, w, None, 1e-5, y, 1024, st[0], st[1], stream())
        lce.lce_layer_norm_backward(4000, 1024, lce.BF16, lce.BF16, x, 1024, x, 1024, w, st[0], st[1], dx, 1024, dw, None,
                                    ws, nws, stream())

    calls()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        calls()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    lce.lce_profile_begin()
    calls()
    prof = lce.lce_profile_end()
    assert prof["other"][1] == 3 and prof["other"][0] > 0


def test_rows_beyond_2_to_the_32_bytes():
    """Layer norm, balance loss and selection on the far end of large tensors."""
    from lm_head_linear_chunked_gb300.balance_loss import balance_forward, balance_fused
    from lm_head_linear_chunked_gb300.beam import beam_select
    from lm_head_linear_chunked_gb300.layer_norm import layer_norm_backward, layer_norm_forward
    rows, H = 700000, 4096
    x = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    x[:] = normal((1000, H), 13, torch.bfloat16).repeat(rows // 1000, 1)
    f = layer_norm_forward(x)
    small = layer_norm_forward(x[:1000])
    assert torch.equal(f["y"][-1000:], small["y"]) and torch.equal(f["rstd"][-1000:], small["rstd"])
    d = layer_norm_backward(x, x, None, f["mean"], f["rstd"], want_grad_weight=False, want_grad_bias=False)
    e = layer_norm_backward(x[:1000], x[:1000], None, small["mean"], small["rstd"], want_grad_weight=False,
                            want_grad_bias=False)
    assert torch.equal(d["grad_x"][-1000:], e["grad_x"])
    del f, d
    # groups and beams a gigabyte apart
    flat = x.view(-1)
    z = flat.as_strided((3, 200, 64), (1 << 30, 64, 1))
    experts = z.float().topk(2, dim=-1).indices
    assert torch.equal(balance_forward(z, experts)["group_loss"], balance_forward(z.clone(), experts)["group_loss"])
    a, b = balance_fused(z, experts), balance_fused(z.clone(), experts)
    assert torch.equal(a["grad_logits"], b["grad_logits"]) and torch.equal(a["loss"], b["loss"])
    logits = flat.as_strided((1, 3, 9001), (3 << 30, 1 << 30, 1))
    scores = torch.tensor([[0.0, -0.3, -0.7]], device="cuda")
    got, want = beam_select(logits, scores, 7), beam_select(logits.clone(), scores, 7)
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_broadcast_inputs_and_gradients():
    """Expanded inputs, and gradients that arrive expanded."""
    from lm_head_linear_chunked_gb300.balance_loss import balance_loss
    from lm_head_linear_chunked_gb300.layer_norm import layer_norm
    row = normal((1, 96), 14).requires_grad_(True)
    w = normal(96, 15).requires_grad_(True)
    layer_norm(row.expand(7, 96), w).sum().backward()
    x = row.detach().double().requires_grad_(True)
    v = w.detach().double().requires_grad_(True)
    torch.nn.functional.layer_norm(x.expand(7, 96), (96,), v).sum().backward()
    # sums of 7 x 96 terms of order one in fp32
    assert (row.grad - x.grad).abs().max() <= 7 * 96 * 2.0 ** -20 and (w.grad - v.grad).abs().max() <= 7 * 2.0 ** -18
    z = normal((1, 40, 8), 16).requires_grad_(True)
    both = z.expand(2, 40, 8)
    experts = both.detach().topk(2, dim=-1).indices
    balance_loss(both, experts)[0].backward()
    one = z.grad.clone()
    z.grad = None
    balance_loss(z, experts[:1])[0].backward()
    assert (one - z.grad).abs().max() <= 2.0 ** -20 * z.grad.abs().max()
