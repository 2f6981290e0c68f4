"""The policy loss whose gradient comes from rows kept in shared memory, where a part of a row is above 32 KB."""
import subprocess
import sys
from pathlib import Path

import pytest

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
