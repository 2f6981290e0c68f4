"""Log-probabilities from hidden states where a wait runs out: the kernel leaves nothing behind, whatever it had begun."""
import pytest
import torch

from test_gpu_head import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,width,n", [(5, 64, 200), (5, 40, 700), (5, 64, 40000), (200, 130, 300), (300, 320, 2000), (40, 2500, 200), (300, 2500, 40000)])
def test_a_wait_that_runs_out(pk, cuda_device, rows, width, n):
    # Fewer pieces than the ring has stages, as many, and more; in one segment and in several.
    hidden, weight, tokens = inputs(rows, width, n, torch.bfloat16)
    tokens[rows // 2] = -1
    want = pk.token_logprobs(hidden, tokens, weight=weight, entropy=True)
    live = tokens >= 0
    for entropy in (True, False):
        pk.set_option(pk.OPT_HEAD_WAIT_TEST, 1)
        got = pk.token_logprobs(hidden, tokens, weight=weight, entropy=entropy)
        torch.cuda.synchronize()
        pk.set_option(pk.OPT_HEAD_WAIT_TEST, 0)
        assert got.logprobs[live].isnan().all() and got.logprobs[rows // 2] == 0
        again = pk.token_logprobs(hidden, tokens, weight=weight, entropy=True)
        assert torch.equal(again.logprobs, want.logprobs) and torch.equal(again.entropies, want.entropies)
