"""Calls that are captured into a graph as the first of their process."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parent.parent
CODE = """
import sys
sys.path.insert(0, {root!r})
import torch
import streaming_selection_primitive_gb300 as pk
rows = 4000
z = torch.randn(rows, 512, device="cuda").bfloat16()
h = z[:, :64].contiguous()
t = torch.zeros(rows, dtype=torch.int64, device="cuda")
one, o = torch.ones(rows, device="cuda"), torch.tensor([0, rows // 2, rows], device="cuda")
noise = torch.ones(rows, 512, device="cuda")
calls = {{"head": lambda: pk.token_logprobs(h, t, weight=h).logprobs, "logprobs": lambda: pk.token_logprobs(z, t).logprobs,
         "policy": lambda: pk.policy_loss(z, t, -6 * one, one, gradient=True).grad_logits, "preference": lambda: pk.preference_loss(z, t, o).slopes,
         "route": lambda: pk.route(z[:, :128], 4).gates, "sample": lambda: pk.sample_tokens(z, noise)[1]}}
call = calls[{call!r}]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(got, call())
"""


@pytest.mark.parametrize("call", ["head", "logprobs", "policy", "preference", "route", "sample"])
def test_first_call(pk, cuda_device, call):
    done = subprocess.run([sys.executable, "-c", CODE.format(root=str(ROOT), call=call)], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
