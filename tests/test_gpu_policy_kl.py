"""The policy loss's KL term where the policy is next to its reference, as in the first steps from it."""
import numpy as np
import pytest
import torch

from logprob_checks import as_numpy, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("apart", [0.0, 1e-7, 1e-5, 1e-3, 0.1, 0.249, 0.3, 5.0])
@pytest.mark.parametrize("gradient", [False, True])
def test_kl_is_not_negative_and_keeps_its_precision(pk, cuda_device, apart, gradient):
    # A call a token, so that each term is seen: by the float32 differences that the kernel has, exactly.  The series is off
    # by seven roundings (2^-21.2), the difference by half a step of e <= 8.4 kl (from q = 0.25 on; 2^-20.9) and expm1's own unit.
    logits, tokens, g = make(24, 300, torch.float32)
    lp = pk.token_logprobs(logits, tokens).logprobs
    ref = lp + apart * (2 * torch.rand(24, generator=g, device=cuda_device) - 1)
    ref[0], ref[1], ref[2] = lp[0], lp[1] + apart, lp[2] - apart
    one = torch.ones(1, device=cuda_device)
    for r in range(24):
        at = slice(r, r + 1)
        got = pk.policy_loss(logits[at], tokens[at], lp[at], one, ref_logprobs=ref[at], kl=1.0, gradient=gradient)
        q = np.longdouble(as_numpy(ref[at] - got.logprobs)[0])  # (exact: they are next to one another, or apart by a float32 step)
        want = float(np.expm1(q) - q if abs(q) > 1e-3 else q * q / 2 + q ** 3 / 6 + q ** 4 / 24 + q ** 5 / 120)
        kl = got.kl.item()
        assert kl >= 0 and abs(kl - want) <= 2.0 ** -19 * want, (r, q, kl, want)
