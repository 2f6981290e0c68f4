"""Rows whose largest logits lie on both sides of the border at which a row's exponents are taken another way
(|m| log2(e) / T = 2^20): which side a part of a row is on must not show in what the parts give together."""
import numpy as np
import pytest
import torch

from oracle import logprobs as ref
from logprob_checks import as_numpy, close, gradient_error, row_error, sizes
from test_gpu_logprobs import check

pytestmark = pytest.mark.gpu

BORDER = 2.0 ** 20 / np.log2(np.e)


def rows_about_the_border(T, sign, n, rows=8, seed=0):
    # Rows that rise or fall through the border, by 3 T about it with 1 T of noise: a row's maximum grows past it as the
    # row is read, and parts that end on either side are joined, each with mass.
    rng = np.random.default_rng(seed + n)
    ramp = 1.5 * np.linspace(-1, 1, n) * np.where(np.arange(rows) % 2, -1, 1)[:, None]
    z = sign * BORDER + ramp + rng.random((rows, n)) - 0.5
    return torch.from_numpy(T * z).float().cuda(), torch.from_numpy(rng.integers(0, n, rows)).cuda()


@pytest.mark.parametrize("T", [1.0, 1e-5, 300.0])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n", [2, 50, 301, 6001, 70001, 300_000])
def test_from_logits(pk, cuda_device, n, sign, T):
    T = float(np.float32(T))
    logits, tokens = rows_about_the_border(T, sign, n)
    check(pk, logits, tokens, T)
    check(pk, logits, tokens, T, entropy=False)


@pytest.mark.parametrize("values,T", [((726817.3, 726817.56), 1.0), ((7.268173, 7.2681756), 1e-5), ((-726817.56, -726817.3), 1.0)])
@pytest.mark.parametrize("n", [2, 3, 40, 6000, 40000])
def test_two_logits(pk, cuda_device, n, values, T):
    # By hand: log-probabilities of two logits that differ by d are -log(1 + exp(-+d / T)).
    T = float(np.float32(T))
    for a, b in ((0, n - 1), (n - 1, 0)):
        z = torch.full((2, n), -float("inf"), device=cuda_device)
        z[:, a], z[:, b] = values
        r = pk.token_logprobs(z, torch.tensor([a, b], device=cuda_device), temperature=T)
        d = (z[0, b].double() - z[0, a].double()).item() / T
        want = np.array([-np.log1p(np.exp(d)), -np.log1p(np.exp(-d))])
        close(as_numpy(r.logprobs), want, row_error(1.0, abs(d), want))


@pytest.mark.parametrize("n", [50, 9001, 40000])
def test_policy_gradient(pk, cuda_device, n):
    # All ratios 1, nothing clipped: the loss is -mean A, its slopes -A / rows.
    logits, tokens = rows_about_the_border(1.0, 1, n)
    l, t = as_numpy(logits), tokens.cpu().numpy()
    lp, _ = ref.logprobs(l, t)
    old = torch.from_numpy(lp).float().cuda()
    A = torch.linspace(-1, 1, len(l), device=cuda_device)
    r = pk.policy_loss(logits, tokens, old, A, gradient=True)
    x, mean = sizes(l, 1.0)
    off = row_error(mean, np.take_along_axis(x, t[:, None], 1)[:, 0], lp)
    close(as_numpy(r.logprobs), lp, off)
    slope = -as_numpy(A) / len(l) * np.exp(lp - as_numpy(old))
    want = ref.gradient(l, t, 1.0, slope)
    p = np.exp(-x) / np.exp(-x).sum(1, keepdims=True)
    moved = (np.abs(slope) * 2 * (off + 2.0 ** -22))[:, None] * (p + (np.arange(n) == t[:, None]))
    close(as_numpy(r.grad_logits), want, gradient_error(l, 1.0, slope, None, want, torch.float32) + moved)


@pytest.mark.parametrize("sign", [1, -1])
def test_from_hidden_states(pk, cuda_device, sign):
    # Logits 726816.5 .. 726818.25 in steps of 0.25: products and sums that float32 (and 23 bits of it) hold exactly.
    g = torch.Generator(device=cuda_device).manual_seed(1)
    n = 3000
    weight = torch.zeros((n, 8), device=cuda_device)
    weight[:, 0] = 709 * sign
    weight[:, 1] = (800.5 + 0.5 * torch.randint(0, 2, (n,), generator=g, device=cuda_device)) * sign
    weight[:, 2] = 0.25 * torch.randint(0, 5, (n,), generator=g, device=cuda_device) * sign
    hidden = torch.zeros((40, 8), device=cuda_device)
    hidden[:, 0], hidden[:, 1], hidden[:, 2] = 1024, 1, 1
    hidden[20:, 2] = 0
    tokens = torch.randint(n, (40,), generator=g, device=cuda_device)
    z = as_numpy(hidden) @ as_numpy(weight).T
    assert (z == z.astype(np.float32)).all() and np.abs(z).min() < BORDER < np.abs(z).max()
    lp, H = ref.logprobs(z, tokens.cpu().numpy())
    x, mean = sizes(z, 1.0)
    at = np.take_along_axis(x, tokens.cpu().numpy()[:, None], 1)[:, 0]
    for entropy in (True, False):
        r = pk.token_logprobs(hidden.half(), tokens, weight=weight.half(), entropy=entropy)
        close(as_numpy(r.logprobs), lp, row_error(mean, at, lp))
    r = pk.token_logprobs(hidden.half(), tokens, weight=weight.half(), entropy=True)
    close(as_numpy(r.entropies), H, row_error(mean, value=H) + 2.0 ** -18 * mean)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [40, 301, 9001])
@pytest.mark.parametrize("h", [1e20, 1e27, 1e33])
def test_masked_logits_under_large_slopes(pk, cuda_device, dtype, n, h):
    # A masked element has the gradient 0 however large its row's slope by the entropy is.
    rng = np.random.default_rng(n)
    logits = torch.from_numpy(rng.normal(size=(6, n))).to(dtype).cuda()
    logits[:, n // 3: n // 2] = -float("inf")
    tokens = torch.full((6,), n - 1, device=cuda_device)
    r = pk.token_logprobs(logits, tokens, entropy=True)
    dh = torch.full((6,), h, device=cuda_device)
    got = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=0 * dh, grad_entropies=dh)
    assert (got[:, n // 3: n // 2] == 0).all() and not got.isnan().any()
    if dtype != torch.float16:  # (beyond what it holds)
        l, t = as_numpy(logits), tokens.cpu().numpy()
        zero, h64 = np.zeros(6), as_numpy(dh)
        want = ref.gradient(l, t, 1.0, zero, h64)
        # (the mean of x as log s - H: 2^-21 of their sizes, as in the test of masked logits at all temperatures)
        x, _ = sizes(l, 1.0)
        p = np.where(np.isfinite(l), np.exp(-x), 0.0)
        p = p / p.sum(1, keepdims=True)
        off = gradient_error(l, 1.0, zero, h64, want, dtype) + h * p * 2.0 ** -21 * 2 * np.log(n)
        close(as_numpy(got), want, off)
