"""A small mixture-of-experts language model, trained and then asked.

The operators around the LM head as a program uses them together:

* training: `LayerNorm` in front of the head, `linear_cross_entropy` for the
  head's loss, `balance_loss` as the mixture's second loss term;
* answering: the head's logits, `beam_select` for each step, `beam_reorder`
  for what the beams carry along.

The model sees one token and has to say the next of the sequence
t -> (5 t + 17) mod V; a few experts per token do the work.  Needs a GB300:

    python examples/train_and_answer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lm_head_linear_chunked_gb300.balance_loss import balance_loss  # noqa: E402
from lm_head_linear_chunked_gb300.beam import beam_reorder, beam_select  # noqa: E402
from lm_head_linear_chunked_gb300.chunk_loss import linear_cross_entropy  # noqa: E402
from lm_head_linear_chunked_gb300.layer_norm import LayerNorm  # noqa: E402

VOCAB, HIDDEN, EXPERTS, SLOTS = 512, 128, 8, 2


def follows(token):
    """The token that comes after `token`."""
    return (5 * token + 17) % VOCAB


class Model(torch.nn.Module):
    def __init__(self):
        super().__init__()
        bf16 = {"dtype": torch.bfloat16, "device": "cuda"}
        self.embedding = torch.nn.Embedding(VOCAB, HIDDEN, **bf16)
        self.router = torch.nn.Linear(HIDDEN, EXPERTS, bias=False, device="cuda")
        self.up = torch.nn.Parameter(torch.randn(EXPERTS, HIDDEN, 2 * HIDDEN, **bf16) * HIDDEN ** -0.5)
        self.down = torch.nn.Parameter(torch.randn(EXPERTS, 2 * HIDDEN, HIDDEN, **bf16) * (2 * HIDDEN) ** -0.5)
        self.norm = LayerNorm(HIDDEN, device="cuda")  # fp32 weight and bias beside bf16 hidden states
        self.head = torch.nn.Linear(HIDDEN, VOCAB, bias=False, **bf16)

    def forward(self, tokens: torch.Tensor):
        """(normed hidden states, router logits, experts of each token) of tokens [N]."""
        h = self.embedding(tokens)
        router = self.router(h.float())
        gates, experts = router.softmax(-1).topk(SLOTS, dim=-1)
        share = torch.zeros_like(router).scatter(1, experts, gates).to(h.dtype)
        # (a toy: every expert sees every token, and the shares pick)
        work = torch.einsum("nh,ehf->enf", h, self.up).relu()
        h = h + torch.einsum("enf,efh,ne->nh", work, self.down, share)
        return self.norm(h), router, experts


def train(model: Model, steps: int, batch: int = 2048):
    """[(loss, balance)] of each step."""
    optimizer = torch.optim.AdamW(model.parameters(), lr=4e-3, weight_decay=0.0)
    generator = torch.Generator(device="cuda").manual_seed(1)
    said = []
    for _ in range(steps):
        tokens = torch.randint(VOCAB, (batch,), device="cuda", generator=generator)
        labels = follows(tokens)
        padding = torch.rand(batch, device="cuda", generator=generator) < 0.1
        hidden, router, experts = model(tokens)
        loss = linear_cross_entropy(hidden, model.head.weight, labels.masked_fill(padding, -100))
        balance, _counts = balance_loss(router, experts, ~padding)
        optimizer.zero_grad()
        (loss + 0.01 * balance).backward()
        optimizer.step()
        said.append(torch.stack((loss.detach(), balance.detach())))
    return torch.stack(said).tolist()


@torch.no_grad()
def answer(model: Model, first: torch.Tensor, beams: int, length: int, end: int = -1):
    """(tokens [items, beams, length], scores [items, beams]) that follow the tokens `first` [items]."""
    items = first.shape[0]
    scores = torch.full((items, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0.0  # before the first step the beams are one
    tokens = first[:, None].expand(items, beams)
    finished = torch.zeros((items, beams), dtype=torch.bool, device="cuda")
    # what a beam carries: its tokens so far, in one of two buffers
    history, other = (torch.zeros((items * beams, length), dtype=torch.int64, device="cuda") for _ in range(2))
    for step in range(length):
        hidden = model(tokens.reshape(-1))[0]
        logits = model.head(hidden).view(items, beams, VOCAB)
        best = beam_select(logits, scores, finished=finished, pad_token=max(end, 0), eos_token=max(end, 0) if end >= 0 else None)
        if step:  # only the part that is written moves
            beam_reorder([history[:, :step]], best["parents"], out=[other[:, :step]])
        history, other = other, history
        scores, tokens = best["scores"], best["tokens"]
        finished = best.get("finished", finished)
        history[:, step] = tokens.reshape(-1)
    return history.view(items, beams, length), scores


def main(steps: int = 150):
    torch.manual_seed(0)
    model = Model()
    said = train(model, steps)
    for step in sorted({0, steps // 2, steps - 1}):
        print(f"step {step}: loss {said[step][0]:.4f}, balance {said[step][1]:.4f}")
    first = torch.tensor([3, 100, 511], device="cuda")
    tokens, scores = answer(model, first, beams=4, length=8)
    right = []
    for i, t in enumerate(first.tolist()):
        want = []
        for _ in range(tokens.shape[2]):
            t = follows(t)
            want.append(t)
        right.append(tokens[i, 0].tolist() == want)
        print(f"{first[i].item()} -> {tokens[i, 0].tolist()} (score {scores[i, 0].item():.3f}, "
              f"{'right' if right[-1] else 'expected ' + str(want)})")
    return said, right


if __name__ == "__main__":
    main()
