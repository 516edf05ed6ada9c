"""The operators around the head together: the example program trains and
answers; its beams agree with a search over all sequences in float64; and a
training step's gradients, recorded into a CUDA graph, have the eager bits."""
import importlib.util
import os

import pytest
import torch

from tests.op_util import normal

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_and_answer", os.path.join(ROOT, "examples", "train_and_answer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_it_learns_and_answers(example):
    said, right = example.main(150)
    assert said[0][0] > 5.0 and said[-1][0] < 0.5 * said[0][0]
    assert all(0.9 < b < 4.5 for _, b in said)  # 1 is even; all slots on two of eight experts give 4
    assert all(right)


def test_beams_against_all_sequences(example):
    """With as many beams as sequences can matter, the best are those of a search over all of them."""
    torch.manual_seed(3)
    model = example.Model()
    first = torch.tensor([7, 450], device="cuda")
    length, beams = 2, 64
    tokens, scores = example.answer(model, first, beams, length)
    with torch.no_grad():
        every = torch.arange(example.VOCAB, device="cuda")
        table = torch.log_softmax(model.head(model(every)[0]).double(), dim=-1)  # [token, next]
    for i, t in enumerate(first.tolist()):
        total = (table[t][:, None] + table).reshape(-1)
        best = total.topk(8)
        # the 8 best of all pairs start with one of the 64 best first tokens
        assert bool((table[t][best.indices // example.VOCAB] >= table[t].topk(beams).values[-1]).all())
        assert torch.allclose(scores[i, :8].double(), best.values, rtol=0, atol=1e-4)
        got = tokens[i, :8, 0] * example.VOCAB + tokens[i, :8, 1]
        near = (best.values[1:] - best.values[:-1]).abs() < 1e-4
        if not bool(near.any()):
            assert torch.equal(got, best.indices)


def test_an_ended_beam_stays(example):
    torch.manual_seed(4)
    model = example.Model()
    first = torch.tensor([9], device="cuda")
    tokens, scores = example.answer(model, first, 6, 5)
    end = int(tokens[0, 0, 0])
    ended, ended_scores = example.answer(model, first, 6, 5, end)
    rows = [r for r in ended[0].tolist() if end in r]
    assert rows and all(set(r[r.index(end):]) == {end} for r in rows)
    assert bool((ended_scores[0, 1:] <= ended_scores[0, :-1]).all())


def test_a_training_step_in_a_graph():
    from lm_head_linear_chunked_gb300.balance_loss import balance_loss
    from lm_head_linear_chunked_gb300.layer_norm import layer_norm
    x = normal((300, 256), 1, torch.bfloat16).requires_grad_(True)
    w = normal(256, 2, mean=1.0, std=0.1).requires_grad_(True)
    b = normal(256, 3, std=0.1).requires_grad_(True)
    z = normal((2, 300, 16), 4).requires_grad_(True)
    experts = z.detach().topk(2, dim=-1).indices
    c = normal((300, 256), 5, torch.bfloat16)

    def step():
        y = layer_norm(x, w, b)
        balance, counts = balance_loss(z, experts)
        return (y.detach(), balance.detach(), counts,
                *torch.autograd.grad((y * c).sum().float() + balance, (x, w, b, z)))

    ref = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, ref):
            assert torch.equal(got, want)
