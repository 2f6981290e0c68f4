"""A small mixture-of-experts language model, trained and sampled with the library's selections.

The tokens come from a random table: each has one successor, followed nine times
in ten (otherwise any token comes).  The model is an embedding, one layer whose
feed-forward network is split into experts, and an output matrix.  Each step

* routes the batch's tokens (``route``): the experts' work is cut up by its
  counts, their outputs are weighted by its gates, and its balance loss is added
  to the model's; the gradient of both comes back through ``route_backward``;
* continues, at the end, a batch of sequences token by token
  (``sample_tokens``, under top-k, top-p and the temperature).

It prints the loss, the balance loss and the share of sampled tokens that
follow the table as one JSON object.

    python -m streaming_selection_primitive_gb300.mixture --steps 200
"""
from __future__ import annotations

import argparse
import json

import torch

import streaming_selection_primitive_gb300 as pk


class Mixture(torch.nn.Module):
    def __init__(self, vocab: int, width: int, experts: int, k: int):
        super().__init__()
        self.k = k
        self.embed = torch.nn.Embedding(vocab, width)
        self.router = torch.nn.Linear(width, experts, bias=False)
        self.up = torch.nn.Parameter(torch.randn(experts, width, 4 * width) * width ** -0.5)
        self.down = torch.nn.Parameter(torch.randn(experts, 4 * width, width) * (4 * width) ** -0.5)
        self.out = torch.nn.Linear(width, vocab, bias=False)

    def forward(self, tokens):
        """Logits of each token's successor, and the routing."""
        x = self.embed(tokens)
        r = pk.route(self.router(x), self.k)
        slots = torch.argsort(r.experts.flatten(), stable=True)  # (token, slot) pairs, expert after expert
        row = slots // self.k
        parts = zip(torch.split(x[row], r.counts.tolist()), self.up, self.down)
        y = torch.cat([torch.relu(part @ up) @ down for part, up, down in parts])
        x = x.index_add(0, row, y * r.gates.flatten()[slots, None])
        return self.out(x), r


def successors(table, tokens, generator):
    """What follows the tokens: nine times in ten the table's, otherwise any."""
    any_token = torch.randint(len(table), tokens.shape, generator=generator, device=tokens.device)
    follow = torch.rand(tokens.shape, generator=generator, device=tokens.device) < 0.9
    return torch.where(follow, table[tokens], any_token)


def train(model, table, steps: int, batch: int, balance: float, generator):
    """(cross entropy, balance loss) of each step."""
    optimizer = torch.optim.Adam(model.parameters(), lr=3e-3)
    history = []
    for _ in range(steps):
        tokens = torch.randint(len(table), (batch,), generator=generator, device=table.device)
        logits, r = model(tokens)
        loss = torch.nn.functional.cross_entropy(logits, successors(table, tokens, generator))
        optimizer.zero_grad(set_to_none=True)
        (loss + balance * r.loss).backward()
        optimizer.step()
        history.append((loss.detach(), r.loss.detach()))
    return [(a.item(), b.item()) for a, b in history]


@torch.no_grad()
def generate(model, first, length: int, generator, *, temperature=0.8, top_k=50, top_p=0.95):
    """(tokens, log-probabilities) of `length` further tokens of each sequence."""
    tokens, logprobs = [first], []
    for _ in range(length):
        logits, _ = model(tokens[-1])
        noise = torch.empty_like(logits, dtype=torch.float32).exponential_(generator=generator)
        token, logprob = pk.sample_tokens(logits, noise, temperature=temperature, top_k=top_k, top_p=top_p)
        tokens.append(token)
        logprobs.append(logprob)
    return torch.stack(tokens, 1), torch.stack(logprobs, 1)


def run(steps=200, batch=2048, vocab=512, width=64, experts=16, k=2, balance=0.01, sequences=32, length=32, seed=0) -> dict:
    device = torch.device("cuda")
    generator = torch.Generator(device=device).manual_seed(seed)
    torch.manual_seed(seed)
    model = Mixture(vocab, width, experts, k).to(device)
    table = torch.randperm(vocab, generator=generator, device=device)
    history = train(model, table, steps, batch, balance, generator)
    tokens, logprobs = generate(model, torch.arange(sequences, device=device) % vocab, length, generator)
    return {
        "steps": steps,
        "loss": [history[0][0], history[-1][0]],
        "balance_loss": [history[0][1], history[-1][1]],
        "followed": (table[tokens[:, :-1]] == tokens[:, 1:]).float().mean().item(),
        "mean_logprob": logprobs.mean().item(),
    }


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--batch", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--k", type=int, default=2)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    print(json.dumps(run(a.steps, a.batch, experts=a.experts, k=a.k, seed=a.seed)))


if __name__ == "__main__":
    main()
