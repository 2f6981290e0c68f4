"""A small mixture-of-experts language model, trained and sampled with the library's selections.

The tokens come from a random table: each has one successor, followed nine times
in ten (otherwise any token comes).  The model is an embedding, one layer whose
feed-forward network is split into experts, and an output matrix.  Each step

* routes the batch's tokens (``route``): the experts' work is cut up by its
  counts, their outputs are weighted by its gates, and its balance loss is added
  to the model's; the gradient of both comes back through ``route_backward``;
* continues, at the end, a batch of sequences token by token
  (``sample_tokens``, under top-k, top-p and the temperature).

With ``--policy-steps`` and ``--preference-steps`` the trained model is trained on
by its own samples: a token is rewarded where it follows the table.  Policy steps (the later ones)
continue sequences, take the advantage of each token over its group's mean
reward, and the clipped policy loss with a KL term to the model as it was
(``policy_loss``; the reference's log-probabilities come straight from its hidden
states, ``token_logprobs`` with a weight).  Preference steps continue each sequence
twice and prefer the continuation that followed the table more often
(``preference_loss``); where both did equally often neither counts.

It prints the loss, the balance loss and the share of sampled tokens that
follow the table as one JSON object.

    python -m streaming_selection_primitive_gb300.mixture --steps 200 --policy-steps 20 --preference-steps 20
"""
from __future__ import annotations

import argparse
import copy
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

    def hidden(self, tokens):
        """What the output matrix makes each token's successor from, and the routing."""
        x = self.embed(tokens)
        r = pk.route(self.router(x), self.k)
        slots = torch.argsort(r.experts.flatten(), stable=True)  # (token, slot) pairs, expert after expert
        row = slots // self.k
        parts = zip(torch.split(x[row], r.counts.tolist()), self.up, self.down)
        y = torch.cat([torch.relu(part @ up) @ down for part, up, down in parts])
        return x.index_add(0, row, y * r.gates.flatten()[slots, None]), r

    def forward(self, tokens):
        """Logits of each token's successor, and the routing."""
        x, r = self.hidden(tokens)
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


def answers(model, table, first, length: int, generator, temperature):
    """Continuations without filters, flat: (inputs, tokens, log-probabilities, whether each follows the table)."""
    tokens, logprobs = generate(model, first, length, generator, temperature=temperature, top_k=0, top_p=1.0)
    inputs, outputs = tokens[:, :-1].flatten(), tokens[:, 1:].flatten()
    return inputs, outputs, logprobs.flatten(), (table[inputs] == outputs).float()


@torch.no_grad()
def reference_logprobs(reference, inputs, tokens, temperature):
    """The reference model's log-probabilities: its head runs in bfloat16, and its logits are never in memory."""
    x, _ = reference.hidden(inputs)
    return pk.token_logprobs(x.bfloat16(), tokens, weight=reference.out.weight.bfloat16(), temperature=temperature).logprobs


def policy_steps(model, table, steps: int, generator, *, groups=32, group=8, length=16, temperature=1.0, kl=0.02, updates=2):
    """(mean reward, loss, KL) of each step."""
    reference = copy.deepcopy(model)
    optimizer = torch.optim.Adam(model.parameters(), lr=1e-3)
    history = []
    for _ in range(steps):
        first = torch.randint(len(table), (groups,), generator=generator, device=table.device).repeat_interleave(group)
        inputs, tokens, old, reward = answers(model, table, first, length, generator, temperature)
        mean = reward.view(groups, group * length).mean(1).repeat_interleave(group * length)
        ref = reference_logprobs(reference, inputs, tokens, temperature)
        for _ in range(updates):  # the second one with ratios other than 1
            logits, _ = model(inputs)
            r = pk.policy_loss(logits, tokens, old, reward - mean, ref_logprobs=ref, temperature=temperature, kl=kl, entropy=0.001)
            optimizer.zero_grad(set_to_none=True)
            r.loss.backward()
            optimizer.step()
        history.append((reward.mean(), r.loss.detach(), r.kl))
    return [tuple(v.item() for v in step) for step in history]


def preferred(inputs, tokens, reward, pairs: int, length: int):
    """The better continuation of each two first: (inputs, tokens, whether each pair has one).  Of two that score the
    same neither is preferred: their tokens are left out (-1), so that no gradient comes from them."""
    score = reward.view(pairs, 2, length).sum(2)
    order = torch.argsort(-score, dim=1, stable=True)[:, :, None].expand(pairs, 2, length)
    inputs, tokens = (torch.gather(t.view(pairs, 2, length), 1, order) for t in (inputs, tokens))
    apart = score[:, 0] != score[:, 1]
    return inputs.flatten(), torch.where(apart[:, None, None], tokens, -1).flatten(), apart


def preference_steps(model, table, steps: int, generator, *, pairs=32, length=16, beta=0.2):
    """(loss, mean margin of the pairs that are compared) of each step."""
    reference = copy.deepcopy(model)
    optimizer = torch.optim.Adam(model.parameters(), lr=1e-3)
    offsets = torch.arange(0, 2 * pairs * length + 1, length, device=table.device)
    history = []
    for _ in range(steps):
        first = torch.randint(len(table), (pairs,), generator=generator, device=table.device).repeat_interleave(2)
        inputs, tokens, _, reward = answers(model, table, first, length, generator, 1.0)
        inputs, tokens, apart = preferred(inputs, tokens, reward, pairs, length)
        ref = reference_logprobs(reference, inputs, tokens, 1.0)
        logits, _ = model(inputs)
        r = pk.preference_loss(logits, tokens, offsets, ref_logprobs=ref, beta=beta)
        optimizer.zero_grad(set_to_none=True)
        r.loss.backward()
        optimizer.step()
        history.append((r.loss.detach(), r.margins.sum() / apart.sum().clamp(min=1)))
    return [tuple(v.item() for v in step) for step in history]


def run(steps=200, batch=2048, vocab=512, width=64, experts=16, k=2, balance=0.01, sequences=32, length=32, seed=0,
        policy=0, preference=0) -> dict:
    device = torch.device("cuda")
    generator = torch.Generator(device=device).manual_seed(seed)
    torch.manual_seed(seed)
    model = Mixture(vocab, width, experts, k).to(device)
    table = torch.randperm(vocab, generator=generator, device=device)
    history = train(model, table, steps, batch, balance, generator)
    trained_on = {}
    if preference:  # (first: after policy steps nearly all continuations score the same)
        margins = preference_steps(model, table, preference, generator)
        trained_on["preference_loss"] = [margins[0][0], margins[-1][0]]
        trained_on["margin"] = margins[-1][1]
    if policy:
        rewards = policy_steps(model, table, policy, generator)
        trained_on["reward"] = [rewards[0][0], rewards[-1][0]]
        trained_on["kl"] = rewards[-1][2]
    tokens, logprobs = generate(model, torch.arange(sequences, device=device) % vocab, length, generator)
    return {
        "steps": steps,
        "loss": [history[0][0], history[-1][0]],
        "balance_loss": [history[0][1], history[-1][1]],
        "followed": (table[tokens[:, :-1]] == tokens[:, 1:]).float().mean().item(),
        "mean_logprob": logprobs.mean().item(),
        **trained_on,
    }


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--batch", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--k", type=int, default=2)
    ap.add_argument("--policy-steps", type=int, default=0)
    ap.add_argument("--preference-steps", type=int, default=0)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    print(json.dumps(run(a.steps, a.batch, experts=a.experts, k=a.k, seed=a.seed, policy=a.policy_steps,
                         preference=a.preference_steps)))


if __name__ == "__main__":
    main()
