"""The log-probabilities and losses as they are used: a model sampled, scored and trained on its samples."""
import copy
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def model(pk, cuda_device):
    from streaming_selection_primitive_gb300 import mixture
    torch.manual_seed(3)
    return mixture.Mixture(256, 32, 8, 2).to(cuda_device)


def test_the_model_runs_with_both_losses(pk, cuda_device):
    from streaming_selection_primitive_gb300 import mixture
    got = mixture.run(steps=20, batch=512, vocab=256, width=32, experts=8, k=2, sequences=8, length=8, policy=3, preference=3)
    values = [*got["reward"], got["kl"], *got["preference_loss"], got["margin"]]
    assert all(math.isfinite(v) for v in values) and got["kl"] >= 0
    # Before a step the model is its own reference, whose head alone is rounded: margins about 0, a loss of log 2.
    assert abs(got["preference_loss"][0] - math.log(2)) < 0.05
    plain = mixture.run(steps=20, batch=512, vocab=256, width=32, experts=8, k=2, sequences=8, length=8)
    assert plain["loss"] == got["loss"] and "reward" not in plain


def gradients(model, loss):
    model.zero_grad(set_to_none=True)
    loss.backward()
    return [p.grad.clone() for p in model.parameters() if p.grad is not None]


def test_a_policy_step_against_torch(pk, cuda_device, model):
    # The same step with the loss in torch's own operations, in float64 from the logits on.
    from streaming_selection_primitive_gb300 import mixture
    g = torch.Generator(device=cuda_device).manual_seed(1)
    first = torch.randint(256, (24,), generator=g, device=cuda_device)
    inputs, tokens, old, reward = mixture.answers(model, torch.arange(256, device=cuda_device), first, 6, g, 0.9)
    old = old - 0.4 * torch.rand(len(old), generator=g, device=cuda_device).round() + 0.1  # ratios 0.9 and 1.35
    A = torch.randn(len(old), generator=g, device=cuda_device)
    ref = mixture.reference_logprobs(copy.deepcopy(model), inputs, tokens, 0.9)
    r = pk.policy_loss(model(inputs)[0], tokens, old, A, ref_logprobs=ref, temperature=0.9, kl=0.1, entropy=0.05)
    got = gradients(model, r.loss)
    logp = torch.log_softmax(model(inputs)[0].double() / 0.9, 1)
    lp, H = logp.gather(1, tokens[:, None])[:, 0], -(logp.exp() * logp).sum(1)
    ratio, q = (lp - old).exp(), ref - lp
    loss = (-torch.minimum(ratio * A, ratio.clamp(0.8, 1.2) * A) + 0.1 * (q.exp() - 1 - q) - 0.05 * H).mean()
    want = gradients(model, loss)
    # Logits of float32 with the same rounding on both sides; from there row errors of 2^-16, and the sums of the
    # backward products, which are float32 on both sides (144 terms: 2^-17 of their sizes).
    torch.testing.assert_close(r.loss.double(), loss, rtol=1e-5, atol=1e-5)
    for a, b in zip(got, want):
        torch.testing.assert_close(a, b, rtol=1e-3, atol=2.0 ** -15 * b.abs().max().item())


def test_a_preference_step_against_torch(pk, cuda_device, model):
    g = torch.Generator(device=cuda_device).manual_seed(2)
    inputs = torch.randint(256, (60,), generator=g, device=cuda_device)
    tokens = torch.randint(256, (60,), generator=g, device=cuda_device)
    ref = -5.5 + torch.randn(60, generator=g, device=cuda_device)
    offsets = torch.tensor([0, 10, 25, 40, 60], device=cuda_device)
    r = pk.preference_loss(model(inputs)[0], tokens, offsets, ref_logprobs=ref, beta=0.3, label_smoothing=0.1)
    got = gradients(model, r.loss)
    logp = torch.log_softmax(model(inputs)[0].double(), 1)
    ratio = logp.gather(1, tokens[:, None])[:, 0] - ref
    D = torch.stack([ratio[a:b].sum() for a, b in zip(offsets[:-1].tolist(), offsets[1:].tolist())])
    d = 0.3 * (D[0::2] - D[1::2])
    loss = -(0.9 * torch.nn.functional.logsigmoid(d) + 0.1 * torch.nn.functional.logsigmoid(-d)).mean()
    want = gradients(model, loss)
    torch.testing.assert_close(r.margins.double(), d, rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(r.loss.double(), loss, rtol=1e-4, atol=1e-5)
    for a, b in zip(got, want):
        torch.testing.assert_close(a, b, rtol=1e-3, atol=2.0 ** -15 * b.abs().max().item())


def test_scores_by_all_ways_agree(pk, cuda_device, model):
    # Sampled, taken from the logits, and from the hidden states in float16 (off by the head's rounding alone).
    g = torch.Generator(device=cuda_device).manual_seed(4)
    inputs = torch.randint(256, (50,), generator=g, device=cuda_device)
    with torch.no_grad():
        logits, _ = model(inputs)
        noise = torch.empty_like(logits).exponential_(generator=g)
        tokens, sampled = pk.sample_tokens(logits, noise, temperature=0.7)
        scored = pk.token_logprobs(logits, tokens, temperature=0.7).logprobs
        x, _ = model.hidden(inputs)
        head = model.out.weight.half()
        direct = pk.token_logprobs(x.half(), tokens, weight=head, temperature=0.7).logprobs
        rounded = pk.token_logprobs(x.half().float() @ head.float().t(), tokens, temperature=0.7).logprobs
    torch.testing.assert_close(scored, sampled, rtol=0, atol=1e-4)
    torch.testing.assert_close(direct, rounded, rtol=0, atol=1e-4)
    torch.testing.assert_close(direct, scored, rtol=0, atol=0.05)


def test_a_step_captured_into_a_graph(pk, cuda_device):
    # Loss and gradient without autograd, into tensors that stay: what a captured training step does.
    g = torch.Generator(device=cuda_device).manual_seed(6)
    hidden = torch.randn((64, 128), generator=g, device=cuda_device).bfloat16()
    weight = (torch.randn((4000, 128), generator=g, device=cuda_device) * 0.1).bfloat16()
    tokens = torch.randint(4000, (64,), generator=g, device=cuda_device)
    old, A = -8.3 + torch.zeros(64, device=cuda_device), torch.randn(64, generator=g, device=cuda_device)
    grad = torch.empty((64, 4000), dtype=torch.bfloat16, device=cuda_device)

    def step():
        ref = pk.token_logprobs(hidden, tokens, weight=weight).logprobs
        logits = hidden @ weight.t()
        r = pk.policy_loss(logits, tokens, old, A, ref_logprobs=ref, kl=0.1, gradient=True, out=grad)
        return r.loss, r.kl, grad.t() @ hidden

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        hidden.copy_(torch.randn((64, 128), generator=g, device=cuda_device).bfloat16())
        graph.replay()
        got = [t.clone() for t in out]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_step_with_autograd_captured_into_a_graph(pk, cuda_device):
    g = torch.Generator(device=cuda_device).manual_seed(7)
    hidden = torch.randn((48, 64), generator=g, device=cuda_device)
    first = torch.randn((5000, 64), generator=g, device=cuda_device) * 0.2
    tokens = torch.randint(5000, (48,), generator=g, device=cuda_device)
    old, A = torch.full((48,), -8.6, device=cuda_device), torch.randn(48, generator=g, device=cuda_device)
    offsets = torch.tensor([0, 12, 24, 36, 48], device=cuda_device)

    def step(weight):
        logits = hidden @ weight.t()
        r = pk.policy_loss(logits, tokens, old, A, entropy=0.1)
        loss = r.loss + pk.preference_loss(logits, tokens, offsets).loss + pk.token_logprobs(logits, tokens).logprobs.mean()
        weight.grad = None
        loss.backward()
        return loss.detach()

    leaf = first.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(leaf)
    torch.cuda.current_stream().wait_stream(side)
    leaf.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step(leaf)
    for _ in range(2):
        hidden.copy_(torch.randn((48, 64), generator=g, device=cuda_device))
        graph.replay()
        other = first.clone().requires_grad_()
        want = step(other)
        assert torch.equal(loss, want) and torch.equal(leaf.grad, other.grad)


def test_without_dependent_launches_the_bits_are_the_same(pk, cuda_device):
    g = torch.Generator(device=cuda_device).manual_seed(8)
    for rows, n in ((700, 304), (60, 20000), (2, 500_000)):
        z = torch.randn((rows, n), generator=g, device=cuda_device).bfloat16()
        t = torch.randint(n, (rows,), generator=g, device=cuda_device)
        one = torch.ones(rows, device=cuda_device)
        offsets = torch.tensor([0, rows // 2, rows], device=cuda_device)

        def calls():
            r = pk.token_logprobs(z, t, entropy=True)
            p = pk.policy_loss(z, t, r.logprobs - 0.05, one, ref_logprobs=r.logprobs, kl=0.1, entropy=0.1, gradient=True)
            q = pk.preference_loss(z, t, offsets)
            h = pk.token_logprobs(z[:, :96], t % 96, weight=z[:2, :96].repeat(48, 1))
            return [*r[:3], *p[:10], *q[:5], pk.preference_loss_backward(z, t, q), h.logprobs]

        want = calls()
        pk.set_option(pk.OPT_PDL, 0)
        got = calls()
        pk.set_option(pk.OPT_PDL, 1)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
