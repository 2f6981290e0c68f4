"""The losses and the product where elements lie beyond 2^31 of them, and where rows are very many."""
import pytest
import torch

from logprob_checks import make
from test_gpu_head import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [200, 9000, 140_001, 500_003])
def test_policy_rows_far_apart(pk, cuda_device, n):
    ld = 1 << 30
    store = torch.empty(2 * ld + (1 << 20), dtype=torch.bfloat16, device=cuda_device)
    far = store.as_strided((3, n), (ld, 1))
    small, tokens, g = make(3, n, torch.bfloat16, -(-n // 8) * 8)  # (rows at the same boundaries: the same order of sums)
    A = torch.randn(3, generator=g, device=cuda_device)
    old = pk.token_logprobs(small, tokens).logprobs - 0.1
    far.copy_(small)
    how = dict(kl=0.1, ref_logprobs=old, entropy=0.1)
    want = pk.policy_loss(small, tokens, old, A, gradient=True, **how)
    plain = pk.policy_loss(far, tokens, old, A, **how)
    assert torch.equal(plain.logprobs, pk.policy_loss(small, tokens, old, A, **how).logprobs)
    got = pk.policy_loss(far, tokens, old, A, gradient=True, out=far, **how)
    assert torch.equal(got.loss, want.loss) and torch.equal(far, want.grad_logits)
    far.copy_(small)
    offsets = torch.tensor([0, 1, 3], device=cuda_device)
    r, q = pk.preference_loss(far, tokens, offsets), pk.preference_loss(small, tokens, offsets)
    assert torch.equal(r.margins, q.margins)
    assert torch.equal(pk.preference_loss_backward(far, tokens, r, out=far), pk.preference_loss_backward(small, tokens, q))


def test_hidden_states_far_apart(pk, cuda_device):
    hidden, weight, tokens = inputs(3, 72, 40, torch.bfloat16)
    want = pk.token_logprobs(hidden, tokens, weight=weight, entropy=True)
    store = torch.empty((1 << 31) + (1 << 20), dtype=torch.bfloat16, device=cuda_device)
    for of in ("hidden", "weight"):
        a, ld = (hidden, 1 << 30) if of == "hidden" else (weight, 1 << 25)
        far = store.as_strided(a.shape, (ld, 1))
        far.copy_(a)
        got = pk.token_logprobs(far if of == "hidden" else hidden, tokens, weight=far if of == "weight" else weight, entropy=True)
        assert torch.equal(got.logprobs, want.logprobs) and torch.equal(got.entropies, want.entropies)


def test_very_many_rows(pk, cuda_device):
    # Against torch in float64; a log-probability is off by 2^-18 at most, and the sums' own rounding is nothing beside that.
    rows, n = (1 << 22) + 5, 6
    logits, tokens, g = make(rows, n, torch.float32, left_out=0.1)
    lp = torch.log_softmax(logits.double(), 1).gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    live = tokens >= 0
    old, A = (lp - 0.05).float(), torch.randn(rows, generator=g, device=cuda_device)
    for gradient in (False, True):
        r = pk.policy_loss(logits, tokens, old, A, gradient=gradient)
        ratio = (lp - old.double()).exp()
        term = torch.where(live, -torch.minimum(ratio * A, ratio.clamp(0.8, 1.2) * A), 0.0)
        assert abs(r.loss.double() - term.sum() / rows) <= 2.0 ** -17 * A.abs().mean()
        assert (r.logprobs.double() - torch.where(live, lp, 0.0)).abs().max() <= 2.0 ** -17
        if gradient:
            p = torch.softmax(logits.double(), 1)
            p.scatter_add_(1, tokens.clamp(min=0)[:, None], torch.full((rows, 1), -1.0, dtype=torch.float64, device=cuda_device))
            want = torch.where(live, A * ratio / rows, 0.0)[:, None] * p
            assert (r.grad_logits.double() - want).abs().max() <= 2.0 ** -16 * A.abs().max() / rows
            assert (r.grad_logits[~live] == 0).all()
    pairs = (rows - 5) // 8
    offsets = torch.arange(0, 2 * pairs + 1, device=cuda_device) * 4 + 2
    r = pk.preference_loss(logits, tokens, offsets, beta=0.3)
    D = torch.where(live, lp, 0.0)[2:-3].view(pairs, 2, 4).sum(2)
    margins = 0.3 * (D[:, 0] - D[:, 1])
    assert (r.margins.double() - margins).abs().max() <= 0.3 * 8 * 2.0 ** -17
    assert abs(r.loss.double() - torch.nn.functional.softplus(-margins).mean()) <= 0.3 * 8 * 2.0 ** -17
