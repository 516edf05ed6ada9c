"""The embedding's gradient by the forms of its sort: from 6145 tokens on by digits, of which a vocabulary of 2^20 rows
takes three and one of 2^30 four, with the rows cleared beside the sort or at the end."""
import pytest
import torch

from tests.op_util import DTYPES, normal
from tests.test_gpu_embedding import check_grad, check_named, tokens_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,V,H,dtype", [
    (9000, (1 << 20) + 3, 8, "bf16"),        # three digits, cleared beside them
    (9000, (1 << 20) + 3, 7, "fp16"),
    (7000, (1 << 20) + 3, 264, "bf16"),      # half a gigabyte and more: cleared at the end
    (70000, (1 << 20) + 3, 8, "fp32"),       # more tokens than are cleared for early
    (6145, 60000, 24, "fp32"),               # two, cleared beside them
    (40000, 50257, 65, "bf16"),
])
@pytest.mark.parametrize("gap", [0, 1, 8])
@pytest.mark.parametrize("kind", ["distinct", "few"])
def test_sorted_by_digits(N, V, H, dtype, gap, kind):
    from lm_head_linear_chunked_gb300.embedding import embedding_backward
    t = tokens_of(kind, N, V, 41)
    room = torch.full((V, H + gap), float("nan"), device="cuda", dtype=DTYPES[dtype])
    dy = normal((N, H), 42, DTYPES[dtype])
    got = embedding_backward(dy, t, V, 1.25, out=room[:, :H])
    check_named(got, dy, t, V, 1.25)
    assert bool(room[:, H:].isnan().all())


@pytest.mark.parametrize("spread", [True, False])
def test_four_digits(spread):
    from lm_head_linear_chunked_gb300.embedding import embedding_backward
    N, V = 7000, (1 << 30) + 1
    t = torch.arange(N, device="cuda") * 153391 if spread else tokens_of("few", N, 1000, 43) * 1073741
    out, dy = torch.full((V, 1), float("nan"), device="cuda", dtype=torch.bfloat16), normal((N, 1), 44, torch.bfloat16)
    check_named(embedding_backward(dy, t, V, 1.25, out=out), dy, t, V, 1.25)


@pytest.mark.parametrize("N,V,H", [(9000, (1 << 20) + 3, 8), (9000, 60000, 24)])
def test_replayed_graphs(N, V, H):
    """Two graphs of one call on their own inputs, replayed in turn and with new inputs, give the eager bits."""
    from lm_head_linear_chunked_gb300.embedding import embedding_backward

    def inputs(seed):
        return tokens_of("zipf", N, V, seed), normal((N, H), seed + 1)

    side = torch.cuda.Stream()
    graphs = []
    for seed in (100, 200):
        t, dy = inputs(seed)
        embedding_backward(dy, t, V)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = embedding_backward(dy, t, V)
        graphs.append((graph, t, dy, out))
    for seed in (300, 400, 300):
        new_t, new_dy = inputs(seed)
        want = embedding_backward(new_dy, new_t, V)
        check_grad(want, new_dy, new_t, V, 1.0)
        for _, t, dy, out in graphs:
            t.copy_(new_t)
            dy.copy_(new_dy)
            out.fill_(float("nan"))
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for *_, out in graphs)
