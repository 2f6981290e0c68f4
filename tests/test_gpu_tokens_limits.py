"""sample_tokens at the limits of its lists, cuts and sums, against the definition in float64.

Tolerances are those of test_gpu_tokens.py (its check and inputs are used here).
"""
import numpy as np
import pytest
import torch

from oracle import selections as ref
from test_gpu_tokens import MASS_BLUR, SCORE_BLUR, TYPES, check, inputs

pytestmark = pytest.mark.gpu


def few_threads_hold_the_top(rows, n, dtype, device, threads, vectors, seed):
    """Rows whose largest logits lie in few threads' vectors: element (t + 512 j) VEC + c of thread t.

    A thread's logits are alike and its level is its own, so that the best of `threads` of them bring all that
    these threads hold."""
    logits, noise = inputs(rows, n, dtype, seed, device)
    g = torch.Generator(device=device)
    g.manual_seed(seed + 1)
    vec = 16 // logits.element_size()
    t = torch.randperm(512, generator=g, device=device)[:threads]
    at = ((t[:, None] + 512 * torch.arange(vectors, device=device))[:, :, None] * vec + torch.arange(vec, device=device))
    level = 10.0 + torch.arange(threads, device=device) / threads
    value = level[:, None, None] + torch.rand(at.shape, generator=g, device=device) / threads
    logits[:, at.flatten()] = value.flatten().to(dtype)
    return logits, noise


@pytest.mark.parametrize("rows", [3, 40, 160, 320])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_keys_than_can_be_ranked(pk, cuda_device, rows, dtype):
    # 1024 keys of a slice can be ranked: copies of one value (no choice of a limit leaves fewer), and many
    # distinct values in few threads (a higher limit does).
    n = 40000
    logits, noise = few_threads_hold_the_top(rows, n, dtype, cuda_device, 120, n // (512 * 16 // (4 if dtype == torch.float32 else 2)), 71)
    logits[::3] = torch.where(torch.arange(n, device=cuda_device) % 7 == 3, 20.0, logits[::3].float()).to(dtype)
    at = torch.arange(0, rows, max(1, rows // 10), device=cuda_device)
    for how in ({"k": 1}, {"k": 50}, {"k": 50, "p": 0.7}, {"T": 0.0}, {"min_p": 0.3}):
        args = {"temperature": how.get("T", 1.0), "top_k": how.get("k", 0), "top_p": how.get("p", 1.0), "min_p": how.get("min_p", 0.0)}
        every, _ = pk.sample_tokens(logits, noise, **args)
        got, _ = check(pk, logits[at], noise[at], most_unclear=0.2, **how)
        if "k" in how or "T" in how:
            assert np.array_equal(every[at].cpu().numpy(), got)


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_tokens_at_the_sampled_ceiling(pk, cuda_device, offset):
    # Float32 logits on a grid of 1/8 (the spacing near 2^20), so that the value above which tokens are raced
    # without a list is on the grid too.  Row r's first three logits are r steps below the largest and
    # have the noise to win: token 0 wherever it is kept.
    rows, n, T, p = 48, 40001, 4.0, 0.5
    g = torch.Generator(device=cuda_device)
    g.manual_seed(81)
    store = torch.zeros(rows * n + offset, device=cuda_device)
    logits = store[offset:].view(rows, n)
    steps = torch.randint(0, 65, (n,), generator=g, device=cuda_device)
    steps[100] = 0
    logits.copy_((2.0 ** 20 + 8 - 0.125 * steps.float()).expand(rows, n))
    logits[:, :3] = 2.0 ** 20 + 8 - 0.125 * torch.arange(rows, device=cuda_device)[:, None].float()
    noise = torch.empty((rows, n), device=cuda_device).exponential_(generator=g)
    noise[:, :3] = torch.tensor([1e-30, 1e-29, 1e-28], device=cuda_device)
    got, _ = check(pk, logits, noise, T=T, p=p, most_unclear=0.1)
    # Half of the mass of levels 0 .. 64 that fall by exp(-1/32) each lies above level 18 or so.
    assert (got[:15] == 0).all() and (got[22:] != 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_2_to_the_28(pk, cuda_device, dtype):
    # Logits of 0 at the start of each eighth of the row (a CTA's slice: every thread meets its maximum at
    # once), and otherwise x: the mass is zeros + (n - zeros) exp(x).  A thread adds up 65536 weights below 1.
    n = 1 << 28
    logits = torch.zeros((1, n), dtype=dtype, device=cuda_device)
    g = torch.Generator(device=cuda_device)
    g.manual_seed(91)
    noise = torch.empty((1, n), device=cuda_device).exponential_(generator=g)
    zeros = 8 * 8192
    off = []
    for x in (-0.15234375, -0.203125, -0.5, -1.5546875, -2.5, -3.0):
        logits.view(8, n // 8)[:, 8192:] = x
        mass = zeros + (n - zeros) * np.exp(x)
        for p in (1.0, 0.5):
            token, lp = (t.item() for t in pk.sample_tokens(logits, noise, top_p=p))
            l = logits[0, token].item()
            off.append(abs(lp - (l - np.log(p * mass))) / (1e-5 + 4e-7 * abs(lp)))
            # The token is the best of those that are surely kept, or one at the cut.
            cut = n if p == 1 else int(n * (p - 2.0 ** -12))
            score = logits[0, :cut].double() - noise[0, :cut].double().log()
            assert l - np.log(noise[0, token].double().item()) >= score.max().item() - 2.0 ** -15
            del score
    assert max(off) < 1, off


@pytest.mark.parametrize("rows,k", [(320, 256), (70, 128)])
def test_the_same_call_gives_the_same_bits_past_the_lists(pk, cuda_device, rows, k):
    # More keys reach the limit than can be ranked, twice, and the third limit lets through about as many as can:
    # which of them a limit is taken from must not depend on the order of the threads.  All scores of a row
    # are equal but for their roundings, so that another way through the kernel shows.
    n, threads, vectors = 65536, k + 40, 16 if k == 256 else 32
    logits, _ = few_threads_hold_the_top(rows, n, torch.float32, cuda_device, threads, vectors if rows > 300 else 8, 101)
    logits[:] = logits[torch.arange(rows, device=cuda_device) % 8]
    noise = torch.exp(logits - logits.amax(1, keepdim=True)) * torch.linspace(0.5, 2.0, rows, device=cuda_device)[:, None]
    for how in ({}, {"top_p": 0.99}):
        want = pk.sample_tokens(logits, noise, top_k=k, **how)
        for _ in range(60):
            got = pk.sample_tokens(logits, noise, top_k=k, **how)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1].view(torch.int32), want[1].view(torch.int32))


@pytest.mark.parametrize("n", [2, 9, 700, 40000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_token_without_weight_is_never_given(pk, cuda_device, n, dtype):
    # Beside +inf (or at a temperature near 0) every other logit weighs nothing, also where the noise of the tokens
    # with weight is never ahead.
    inf, nan = float("inf"), float("nan")
    logits, noise = inputs(6, n, dtype, 111, cuda_device)
    at = n // 2
    for r, (q, l) in enumerate([(nan, inf), (inf, inf), (-1.0, inf), (nan, 30.0), (inf, 30.0), (1.0, inf)]):
        logits[r, at], noise[r, at] = l, q
    T = torch.tensor([1.0, 1.0, 1.0, 1e-39, 1e-39, 1.0], device=cuda_device)
    for how in ({}, {"top_k": 5}, {"top_p": 0.9}, {"min_p": 0.01}):
        got, lp = pk.sample_tokens(logits, noise, temperature=T, **how)
        assert (got == at).all() and (lp == 0).all(), how


def cluster_of(rows, n, size, processors):
    """CTAs of a row: up to 8 while they have room at once (two a processor) and each has 16 KB."""
    vec, c = 16 // size, 1
    nbytes = (n + 2 * vec - 2) // vec * 16
    while c < 8 and rows * c * 2 <= 2 * processors and nbytes // (2 * c) >= 16384:
        c *= 2
    return c


def check_some(pk, logits, noise, at, T=1.0, k=0, p=1.0, min_p=0.0):
    """The call over all rows, and the rows `at` against the definition: tokens, and what the others may be."""
    got, lp = pk.sample_tokens(logits, noise, temperature=T, top_k=k, top_p=p, min_p=min_p)
    l, q = logits[at].double().cpu().numpy(), noise[at].double().cpu().numpy()
    numbers = [np.float32(x).item() for x in (p, min_p)]
    may = []
    for i, r in enumerate(at):
        want = ref.tokens_within(l[i], q[i], np.ones(l.shape[1], bool), np.float32(T).item(), k, *numbers, SCORE_BLUR, MASS_BLUR)
        assert got[r].item() in want, (r, got[r].item(), want)
        lo, hi = want[got[r].item()]
        room = 1e-5 + 4e-7 * abs(lo)
        assert lo - room <= lp[r].item() <= hi + room, (r, lp[r].item(), lo, hi)
        may.append(want)
    return got[at], lp[at], may


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("c", [1, 2, 4, 8])
def test_lists_that_clusters_join(pk, cuda_device, c, dtype):
    # Around the 128 keys that a CTA of a cluster may send (256 of a CTA alone): ties across the cut and across the
    # slices' borders, and slices that all hold the same values, so that each sends all that it may.
    processors = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    size, n = dtype.itemsize, 135000 // dtype.itemsize
    vec = 16 // size
    rows = {1: 2 * processors, 2: processors, 4: processors // 2, 8: processors // 4}[c]
    assert cluster_of(rows, n, size, processors) == c
    logits, noise = inputs(rows, n, dtype, 121 + c, cuda_device)
    per = -(-((n + 2 * vec - 2) // vec) // c) * vec  # elements of a slice (rows on the 16-byte boundary)
    logits[::2] = (logits[::2].float() * 8).round().to(dtype) / 8
    logits[1::4] = logits[1::4, :per].repeat(1, c)[:, :n]
    logits[3::8] = torch.sort(logits[3::8], dim=1, descending=True).values
    at = list(range(0, rows, max(1, rows // 12)))[:12] + [1, 3, 5]
    for k in (2, 17, 127, 128, 129, 130, 255, 256, 257):
        check_some(pk, logits, noise, at, k=k)
    for how in ({"k": 128, "p": 0.95}, {"k": 127, "p": 0.9, "min_p": 0.2}, {"p": 0.02}, {"p": 0.3, "T": 0.4}, {"min_p": 0.2}, {"T": 0.0}):
        check_some(pk, logits, noise, at, **how)


@pytest.mark.parametrize("n", [33333, 90001])
def test_rows_shared_out_otherwise_agree_but_for_near_ties(pk, cuda_device, n):
    # The same rows by one, two, four and eight CTAs each: a token that differs is one of several within the
    # scores' or the masses' roundings.
    rows = 320
    logits, noise = inputs(rows, n, torch.float32, 131, cuda_device, spread=0.4)
    at = list(range(0, 12))
    for how in ({"p": 0.9}, {"p": 0.97, "min_p": 0.05}, {"k": 20000, "p": 0.8}, {"k": 100}, {"min_p": 0.1}, {}):
        first = None
        for some in (320, 100, 50, 20):
            got, lp, may = check_some(pk, logits[:some], noise[:some], at, **how)
            if first is None:
                first = got, lp
            for i in range(len(at)):
                if got[i] != first[0][i]:
                    assert len(may[i]) > 1 and first[0][i].item() in may[i]
                else:
                    assert abs(lp[i] - first[1][i]).item() < 2e-5
