"""The policy loss whose gradient comes from rows kept in shared memory, where a part of a row is above 32 KB."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

from test_gpu_policy import check_policy, policy_inputs

pytestmark = pytest.mark.gpu

TESTS = Path(__file__).resolve().parent

# A kernel's limit of shared memory stays as high as a call has set it: in a process of its own, each call here is its
# kernel's first one (types and entropies are kernels of their own).
FIRST_CALLS = """
import sys
sys.path[:0] = [{tests!r}, {root!r}]
import torch
import streaming_selection_primitive_gb300 as pk
from test_gpu_policy import check_policy
for dtype in (torch.float32, torch.bfloat16, torch.float16):
    for entropy in (None, 0.05):
        check_policy(pk, 2, {row} // dtype.itemsize, dtype, entropy=entropy)
"""


@pytest.mark.parametrize("part", [48100, 48640, 49104])
def test_parts_just_below_48_kb_as_the_first_call(pk, cuda_device, part):
    # With the kernel's own shared memory a CTA is above the 48 KB that a launch has without asking.
    code = FIRST_CALLS.format(tests=str(TESTS), root=str(TESTS.parent), row=8 * part)
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


# A part of a row is above 32 KB from 262144 bytes a row on, and the row is kept up to eight parts of 112 KB less the room
# for single elements; behind that it is read twice.
LAST = 8 * (112 * 1024 - 48)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("row", [262144 - 16, 262144, 262144 + 4, 262144 + 16, 8 * 47104, 8 * 48640 + 12, 8 * 49200, 600_004, LAST - 100, LAST, LAST + 4, LAST + 64])
def test_rows_in_eight_large_parts(pk, cuda_device, dtype, row):
    n = row // dtype.itemsize
    check_policy(pk, 2, n, dtype, entropy=None, ld=n + 1, offset=1)  # a row at another place to the 16-byte boundaries than the next
    check_policy(pk, 2, n - 1, dtype, ld=n + 3, offset=5, T=0.8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shift", range(1, 8))
def test_large_parts_into_places_of_any_alignment(pk, cuda_device, dtype, shift):
    n = 300_003 // dtype.itemsize
    logits, tokens, old, A, refs, w, _, _ = policy_inputs(3, n, dtype, left_out=0.3)
    tokens[0], tokens[1] = 0, n - 1
    how = dict(ref_logprobs=refs, weights=w, kl=0.1, entropy=0.1, gradient=True)
    want = pk.policy_loss(logits, tokens, old, A, **how)
    store = torch.full((3 * (n + 5) + 16,), 7.0, dtype=dtype, device=cuda_device)
    out = store[shift:shift + 3 * (n + 5)].view(3, n + 5)[:, :n]
    got = pk.policy_loss(logits, tokens, old, A, out=out, **how)
    assert torch.equal(out, want.grad_logits) and torch.equal(got.loss, want.loss)
    out.fill_(7.0)
    assert (store == 7).all()  # nothing beside it was written
    place = logits.clone()
    pk.policy_loss(place, tokens, old, A, out=place, **how)
    assert torch.equal(place, want.grad_logits)


def test_large_parts_of_many_rows(pk, cuda_device):
    # More clusters than the SMs hold at once, and rows left out among them.
    logits, tokens, old, A, refs, w, _, _ = policy_inputs(130, 151_936, torch.bfloat16, left_out=0.2)
    how = dict(ref_logprobs=refs, weights=w, kl=0.1, entropy=0.05)
    fused = pk.policy_loss(logits, tokens, old, A, gradient=True, **how)
    for rows in torch.arange(130, device=cuda_device).split(13):
        part = pk.policy_loss(logits[rows], tokens[rows], old[rows], A[rows], gradient=True, ref_logprobs=refs[rows], weights=w[rows], kl=0.1, entropy=0.05)
        assert torch.equal(part.grad_logits, fused.grad_logits[rows]) and torch.equal(part.logprobs, fused.logprobs[rows])
    again = pk.policy_loss(logits, tokens, old, A, gradient=True, **how)
    assert torch.equal(again.grad_logits, fused.grad_logits) and torch.equal(again.loss, fused.loss)
