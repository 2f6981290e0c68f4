"""sample_tokens against its definition in float64 (oracle/selections.py).

Tokens have to be equal but where float32 blurs the definition's decision: a
score is x - log q with |x| < 2^7 and so within 2^-16 of its exact value; a
mass is a sum of weights of two ulps and an x error of 2^-22 |x|, |x| < 8 where
the mass is.  Log-probabilities: x carries three roundings (2^-22 |x| with
room), the sum's logarithm the masses' blur and one ulp of a number below 16.
"""
import numpy as np
import pytest
import torch

from oracle import selections as ref

pytestmark = pytest.mark.gpu

SCORE_BLUR, MASS_BLUR = 2.0 ** -15, 2.0 ** -19
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def inputs(rows, n, dtype, seed, device, ld=None, offset=0, spread=2.0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    ld = ld or n
    store = torch.empty(rows * ld + offset, dtype=dtype, device=device).fill_(torch.finfo(dtype).max)
    logits = store[offset:].view(rows, ld)[:, :n]
    logits.copy_(spread * torch.randn((rows, n), generator=g, device=device))
    noise = torch.empty((rows, n), device=device).exponential_(generator=g)
    return logits, noise


def unpack(mask, n):
    words = mask.cpu().numpy().view(np.uint8).reshape(mask.shape[0], -1)
    return np.unpackbits(words, axis=1, bitorder="little")[:, :n].astype(bool)


def check(pk, logits, noise, T=1.0, k=0, p=1.0, min_p=0.0, mask=None, most_unclear=0.02):
    got, lp = pk.sample_tokens(logits, noise, temperature=T, top_k=k, top_p=p, min_p=min_p, mask=mask)
    assert got.dtype == torch.int64 and lp.dtype == torch.float32 and got.shape == lp.shape == (logits.shape[0],)
    again, lp2 = pk.sample_tokens(logits, noise, temperature=T, top_k=k, top_p=p, min_p=min_p, mask=mask)
    assert torch.equal(got, again) and torch.equal(lp.view(torch.int32), lp2.view(torch.int32))
    l, q = logits.double().cpu().numpy(), noise.double().cpu().numpy()
    rows, n = l.shape
    allowed = np.ones((rows, n), bool) if mask is None else unpack(mask, n)
    at = lambda v, r: v[r].item() if isinstance(v, torch.Tensor) else v  # noqa: E731
    got, lp = got.cpu().numpy(), lp.cpu().numpy()
    unclear = 0
    for r in range(rows):
        # float32 parameters, as the call takes them
        want = ref.tokens_within(l[r], q[r], allowed[r], np.float32(at(T, r)).item(), at(k, r), np.float32(at(p, r)).item(),
                                 np.float32(at(min_p, r)).item(), SCORE_BLUR, MASS_BLUR)
        unclear += len(want) > 1
        assert int(got[r]) in want, (r, got[r], want)
        lo, hi = want[int(got[r])]
        if np.isfinite(lo):
            room = 1e-5 + 4e-7 * abs(lo)
            assert lo - room <= lp[r] <= hi + room, (r, lp[r], lo, hi)
        else:
            assert np.isnan(lp[r]) if np.isnan(lo) else lp[r] == lo, (r, lp[r], lo)
    assert unclear <= max(1, most_unclear * rows), unclear
    return got, lp


FILTERS = {
    "none": {}, "greedy": {"T": 0.0}, "k1": {"k": 1}, "k50": {"k": 50}, "k2000": {"k": 2000}, "p.9": {"p": 0.9},
    "p.999 hot": {"p": 0.999, "T": 2.0}, "min_p": {"min_p": 0.05}, "all cold": {"k": 40, "p": 0.8, "min_p": 0.02, "T": 0.5},
    "kp": {"k": 300, "p": 0.95}, "p0": {"p": 0.0},
}


@pytest.mark.parametrize("how", FILTERS)
@pytest.mark.parametrize("dtype", TYPES)
def test_filters(pk, cuda_device, how, dtype):
    logits, noise = inputs(9, 33333, dtype, 5, cuda_device)
    check(pk, logits, noise, **FILTERS[how])


@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 31, 32, 33, 127, 1000, 4097, 65536, 128003, 262145])
@pytest.mark.parametrize("dtype", TYPES)
def test_lengths(pk, cuda_device, n, dtype):
    rows = 5 if n > 1000 else 40
    logits, noise = inputs(rows, n, dtype, n, cuda_device)
    for how in ({}, {"k": 20}, {"p": 0.85}, {"k": 64, "p": 0.7, "min_p": 0.01, "T": 0.8}):
        check(pk, logits, noise, most_unclear=0.05, **how)


@pytest.mark.parametrize("rows,n", [(1, 32768), (1, 500000), (2, 128000), (33, 50001), (160, 20000), (700, 3001), (3000, 130)])
def test_batches(pk, cuda_device, rows, n):
    logits, noise = inputs(rows, n, torch.bfloat16, rows, cuda_device)
    check(pk, logits, noise, k=30, p=0.9)
    check(pk, logits, noise, T=0.9)


@pytest.mark.parametrize("how", ["k2000", "p.9", "p.999 hot", "min_p", "all cold", "kp"])
@pytest.mark.parametrize("dtype,n", [(torch.float32, 9001), (torch.bfloat16, 20004), (torch.float16, 3000)])
def test_more_rows_than_processors(pk, cuda_device, dtype, n, how):
    # Rows that a CTA alone cannot finish are left to clusters.
    logits, noise = inputs(320, n, dtype, 31, cuda_device)
    logits[::7] *= 0.02  # flat: thousands of tokens are kept
    logits[3::31] = float("-inf")
    logits[5, 17] = float("nan")
    g = torch.Generator(device=cuda_device)
    g.manual_seed(2)
    mask = torch.randint(-(1 << 31), 1 << 31, (320, (n + 31) // 32), generator=g, device=cuda_device).to(torch.int32)
    mask[9::40] = 0
    got, lp = check(pk, logits, noise, **FILTERS[how])
    assert (got[3::31] == -1).all() and (lp[3::31] == -np.inf).all() and got[5] == -1 and np.isnan(lp[5])
    got, lp = check(pk, logits, noise, mask=mask, **FILTERS[how])
    assert (got[9::40] == -1).all()


@pytest.mark.parametrize("rows", [30, 76, 320])
@pytest.mark.parametrize("k", [63, 64, 65, 128, 129, 255, 256, 257, 511, 600])
def test_list_lengths(pk, cuda_device, k, rows):
    # Around the lengths where the ranked lists end, with ties across the cut.
    logits, noise = inputs(rows, 6000, torch.float32, k, cuda_device)
    logits[::2] = (logits[::2] * 8).round() / 8
    check(pk, logits, noise, k=k, most_unclear=0.03)
    check(pk, logits, noise, k=k, p=0.97, min_p=0.004, most_unclear=0.03)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 18, 37, 75])
def test_clusters(pk, cuda_device, rows, dtype):
    # 8, 8, 4 and 2 CTAs a row; flat and steep rows, kept tokens side by side or apart.
    logits, noise = inputs(rows, 40009, dtype, 41, cuda_device)
    logits[::3] *= 0.1
    logits[1::5] = torch.sort(logits[1::5], dim=1).values
    for how in ("k2000", "p.9", "p.999 hot", "kp", "min_p", "none"):
        check(pk, logits, noise, most_unclear=0.05, **FILTERS[how])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [3, 40, 160])
def test_rows_that_keep_much(pk, cuda_device, rows, dtype):
    # Tens of thousands of tokens are kept: odd rows, noise off the 16-byte grid, masks, min-p after top-p.
    n = 45001 if rows > 100 else 90001
    logits, noise = inputs(rows, n, dtype, rows, cuda_device, ld=n + 3, offset=1, spread=0.4)
    shifted = torch.cat([noise, noise[:, :1]], 1)[:, 1:]
    g = torch.Generator(device=cuda_device)
    g.manual_seed(3)
    mask = torch.randint(-(1 << 31), 1 << 31, (rows, (n + 31) // 32), generator=g, device=cuda_device).to(torch.int32)
    few = 12  # the definition sorts every row
    for how in ({"p": 0.9}, {"p": 0.97, "min_p": 0.05}, {"p": 0.6, "T": 0.3, "mask": mask}, {"k": 20000, "p": 0.8}, {"min_p": 0.1}):
        m = how.get("mask")
        args = {"temperature": how.get("T", 1.0), "top_k": how.get("k", 0), "top_p": how.get("p", 1.0), "min_p": how.get("min_p", 0.0)}
        all_tokens, all_logprobs = pk.sample_tokens(logits, shifted, mask=m, **args)
        at = torch.arange(0, rows, max(1, rows // few), device=cuda_device)
        got, lp = check(pk, logits[at], shifted[at], most_unclear=0.2,
                        **{**how, **({"mask": m[at].contiguous()} if m is not None else {})})
        # A row's choice does not depend on how many CTAs shared it (its log-probability by the masses' roundings).
        assert (all_tokens[at].cpu().numpy() == got).mean() > 0.8
        assert np.allclose(all_logprobs[at].cpu().numpy()[all_tokens[at].cpu().numpy() == got],
                           lp[all_tokens[at].cpu().numpy() == got], rtol=0, atol=2e-5)


@pytest.mark.parametrize("rows", [2, 160])
def test_noise_extremes_where_much_is_kept(pk, cuda_device, rows):
    n = 40000
    logits, noise = inputs(rows, n, torch.float32, 61, cuda_device, spread=0.1)
    top = logits.argmax(1)
    noise[0, top[0]] = 0.0              # ahead of everything
    noise[1, :] = float("nan")          # never ahead
    noise[1, top[1]] = 5.0
    if rows > 2:
        noise[2, :] = -1.0
        noise[2, top[2]] = float("inf")
        noise[3, top[3]] = 1e-42        # below the normal range: 97 ahead of an ordinary number
        noise[4, ::2] = float("inf")
    for how in ({"p": 0.9}, {"p": 0.9, "min_p": 0.5}, {"k": 30000}):
        got, _ = check(pk, logits[:8], noise[:8], **how)
        for _ in range(2):
            args = {"top_k": how.get("k", 0), "top_p": how.get("p", 1.0), "min_p": how.get("min_p", 0.0)}
            every, _ = pk.sample_tokens(logits, noise, **args)
        want = [0, 1, 3] if rows > 2 else [0, 1]
        assert all(every[r] == top[r] == int(got[r]) for r in want)
        if rows > 2:
            assert every[4] % 2 == 1


def test_rows_far_apart(pk, cuda_device):
    # Offsets of logits and noise past 2^31 elements.
    n, far = 5000, (1 << 30) + 1024
    store = torch.empty(2 * far + n, dtype=torch.bfloat16, device=cuda_device)
    numbers = torch.empty(2 * far + n, device=cuda_device)
    logits, noise = (t.as_strided((3, n), (far, 1)) for t in (store, numbers))
    a, b = inputs(3, n, torch.bfloat16, 51, cuda_device)
    logits.copy_(a)
    noise.copy_(b)
    for how in ({"k": 40}, {"p": 0.95}, {}):
        want = pk.sample_tokens(a, b, top_k=how.get("k", 0), top_p=how.get("p", 1.0))
        got = pk.sample_tokens(logits, noise, top_k=how.get("k", 0), top_p=how.get("p", 1.0))
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        check(pk, a, b, **how)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ld,offset", [(10007, 0), (10008, 0), (10016, 1), (10011, 3), (12000, 8)])
def test_strides_and_alignment(pk, cuda_device, dtype, ld, offset):
    # The store's other places hold the type's largest value: a read outside the row wins.
    logits, noise = inputs(6, 10007, dtype, 3, cuda_device, ld=ld, offset=offset)
    check(pk, logits, noise, p=0.9)
    check(pk, logits, noise[:, :1].expand(6, 10007).contiguous(), k=50)
    check(pk, logits, noise[:1].expand(6, 10007), T=0.7)  # one row of numbers for all
    wide = torch.cat([noise, noise], 1)[:, 1:10008]
    check(pk, logits, wide, min_p=0.03)


def test_parameters_of_each_row(pk, cuda_device):
    rows = 64
    logits, noise = inputs(rows, 20001, torch.bfloat16, 11, cuda_device)
    i = torch.arange(rows, device=cuda_device)
    T = torch.where(i % 8 == 0, 0.0, 0.5 + 0.02 * i)
    k = torch.where(i % 4 == 1, i + 1, torch.where(i % 4 == 2, 0, -3)).to(torch.int32)
    p = torch.where(i % 3 == 0, 0.3 + 0.01 * i, 1.0)
    min_p = torch.where(i % 5 == 0, 0.01 * (1 + i % 7), 0.0)
    check(pk, logits, noise, T=T, k=k, p=p, min_p=min_p)


def test_bad_parameters_of_a_row_are_its_own(pk, cuda_device):
    logits, noise = inputs(6, 1000, torch.float32, 2, cuda_device)
    nan = float("nan")
    T = torch.tensor([1.0, -1.0, nan, 1.0, 1.0, 1.0], device=cuda_device)
    p = torch.tensor([0.9, 0.9, 0.9, nan, 0.9, 2.0], device=cuda_device)
    m = torch.tensor([0.0, 0.0, 0.0, 0.0, nan, -1.0], device=cuda_device)
    got, lp = check(pk, logits, noise, T=T, p=p, min_p=m)
    assert (got[[1, 2, 3, 4]] == -1).all() and np.isnan(lp[[1, 2, 3, 4]]).all() and (got[[0, 5]] >= 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [31, 5000, 70001])
def test_masks(pk, cuda_device, dtype, n):
    rows = 8
    logits, noise = inputs(rows, n, dtype, 7, cuda_device)
    g = torch.Generator(device=cuda_device)
    g.manual_seed(1)
    mask = torch.randint(-(1 << 31), 1 << 31, (rows, (n + 31) // 32), generator=g, device=cuda_device).to(torch.int32)
    mask[0] = 0  # nothing allowed (but for the bits past the end)
    if n % 32:
        mask[0, -1] = -(1 << (n % 32)) if n % 32 < 31 else -(1 << 31)
    mask[1] = -1
    mask[2] = 0
    mask[2, n // 64] = 1 << (n // 2 % 32)  # one token allowed
    # What masked places hold does not matter.
    allowed = torch.from_numpy(unpack(mask, n)).to(cuda_device)
    junk = torch.tensor([float("nan"), float("inf"), torch.finfo(dtype).max], device=cuda_device).to(dtype)
    logits.copy_(torch.where(allowed, logits, junk[torch.arange(n, device=cuda_device) % 3]))
    for how in FILTERS.values():
        got, lp = check(pk, logits, noise, mask=mask, **how)
        assert got[0] == -1 and lp[0] == -np.inf and got[2] == n // 64 * 32 + n // 2 % 32
    wide = torch.cat([mask, mask], 1)[:, :mask.shape[1]]
    check(pk, logits, noise, mask=wide, p=0.9)


@pytest.mark.parametrize("dtype", TYPES)
def test_special_values(pk, cuda_device, dtype):
    n = 3000
    logits, noise = inputs(10, n, dtype, 9, cuda_device)
    inf, low = float("inf"), torch.finfo(dtype).min
    logits[0] = -inf                     # nothing to choose
    logits[1] = low                      # the type's lowest value is a value
    logits[2] = -inf
    logits[2, 77] = low
    logits[3, [5, 900]] = inf            # +inf shares the mass among its copies
    logits[4, 10] = float("nan")
    logits[5, :] = 0.0                   # every token tied
    logits[6, ::2] = -0.0
    logits[6, 1::2] = 0.0                # signed zeros are equal
    logits[7, 100:] = low
    logits[8] = torch.finfo(dtype).max
    for how in ({}, {"k": 7}, {"p": 0.4995}, {"min_p": 0.1}, {"T": 0.0}, {"k": 100, "p": 0.4951, "T": 0.3}):
        got, lp = check(pk, logits, noise, **how)
        assert got[0] == -1 and lp[0] == -inf and got[4] == -1 and np.isnan(lp[4]) and got[2] == 77
        assert got[3] in (5, 900)
    # Ties are kept by lowest index.
    got, _ = check(pk, logits, noise, k=7)
    assert got[5] < 7 and got[6] < 7 and got[8] < 7
    got, _ = check(pk, logits, noise, T=0.0)
    assert got[5] == got[6] == got[8] == 0


def test_temperatures(pk, cuda_device):
    logits, noise = inputs(4, 5000, torch.float32, 21, cuda_device)
    for T in (1e-30, 1e-3, 0.05, 30.0, 1e30, float("inf")):
        check(pk, logits, noise, T=T)
        check(pk, logits, noise, T=T, k=10)
        check(pk, logits, noise, T=T, p=0.70003)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("spread", [0.0, 0.01, 0.3, 20.0])
def test_flat_and_steep_rows(pk, cuda_device, dtype, spread):
    # Flat rows keep tens of thousands of tokens; 16-bit ones hold thousands of copies of a value.
    logits, noise = inputs(4, 90000, dtype, 4, cuda_device, spread=spread)
    check(pk, logits, noise, p=0.9)
    check(pk, logits, noise, k=30000)
    check(pk, logits, noise, k=50000, p=0.5)
    check(pk, logits, noise, min_p=0.3)


def test_sorted_rows(pk, cuda_device):
    # The largest logits side by side, at either end of the row.
    logits, noise = inputs(6, 120000, torch.float32, 8, cuda_device)
    v = torch.sort(logits, dim=1).values
    v[::2] = v[::2].flip(1)
    for how in ({"k": 1000}, {"p": 0.9}, {"p": 0.3}, {"min_p": 0.01}, {}):
        check(pk, v.contiguous(), noise, **how)


def test_noise_extremes(pk, cuda_device):
    logits, noise = inputs(5, 400, torch.float32, 6, cuda_device)
    noise[0, 33] = 0.0            # -log 0 = inf: ahead of everything
    noise[1, :] = float("nan")    # never ahead: the lowest index kept
    noise[2, :200] = -1.0
    noise[3, 7] = float("inf")
    got, _ = check(pk, logits, noise)
    assert got[0] == 33 and got[1] == 0 and got[2] >= 200 and got[3] != 7


@pytest.mark.parametrize("how", [{}, {"k": 12}, {"p": 0.8}, {"min_p": 0.1}])
def test_frequencies(pk, cuda_device, how):
    # One distribution drawn 200,000 times: chi-square against its probabilities.
    n, draws = 40, 200_000
    logits, _ = inputs(1, n, torch.float32, 30, cuda_device, spread=1.0)
    g = torch.Generator(device=cuda_device)
    g.manual_seed(77)
    noise = torch.empty((draws, n), device=cuda_device).exponential_(generator=g)
    args = {"top_k": how.get("k", 0), "top_p": how.get("p", 1.0), "min_p": how.get("min_p", 0.0)}
    got, lp = pk.sample_tokens(logits.expand(draws, n).contiguous(), noise, **args)
    seen = torch.bincount(got, minlength=n).cpu().numpy()
    prob = np.zeros(n)
    prob[got.cpu().numpy()] = np.exp(lp.double().cpu().numpy())
    assert abs(prob.sum() - 1) < 1e-4  # what is seen is everything that is kept
    kept = prob > 0
    chi = ((seen[kept] - draws * prob[kept]) ** 2 / (draws * prob[kept])).sum()
    df = kept.sum() - 1
    assert chi < df + 4.5 * np.sqrt(2 * df) + 12, (chi, df)


def test_streams_outputs_and_graph(pk, cuda_device):
    logits, noise = inputs(16, 40000, torch.bfloat16, 14, cuda_device)
    want, wlp = pk.sample_tokens(logits, noise, top_k=50, top_p=0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, lp = pk.sample_tokens(logits, noise, top_k=50, top_p=0.9, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(lp, wlp)
    out = (torch.empty_like(want), torch.empty_like(wlp))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.sample_tokens(logits, noise, top_k=50, top_p=0.9, out=out)
    other = noise.flip(0).contiguous()
    noise.copy_(other)
    graph.replay()
    want, wlp = pk.sample_tokens(logits, other, top_k=50, top_p=0.9)
    assert torch.equal(out[0], want) and torch.equal(out[1], wlp)
    e, elp = pk.sample_tokens(logits[:0], noise[:0])
    assert e.shape == elp.shape == (0,)


def test_refusals(pk, cuda_device):
    logits, noise = inputs(4, 100, torch.float32, 1, cuda_device)
    with pytest.raises(TypeError):
        pk.sample_tokens(logits.double(), noise)
    with pytest.raises(TypeError):
        pk.sample_tokens(logits.cpu(), noise)
    with pytest.raises(TypeError):
        pk.sample_tokens(logits, noise.half())
    with pytest.raises(ValueError):
        pk.sample_tokens(logits[0], noise[0])
    with pytest.raises(ValueError):
        pk.sample_tokens(logits, noise[:, :50])
    with pytest.raises(ValueError):
        pk.sample_tokens(logits.t(), noise.t().contiguous())
    with pytest.raises(ValueError):
        pk.sample_tokens(logits, noise.t().contiguous().t())
    with pytest.raises(TypeError):
        pk.sample_tokens(logits, noise, top_k=torch.ones(4, device=cuda_device))
    with pytest.raises(ValueError):
        pk.sample_tokens(logits, noise, top_p=torch.ones(3, device=cuda_device))
    with pytest.raises(TypeError):
        pk.sample_tokens(logits, noise, temperature=torch.ones(4))
    with pytest.raises(TypeError):
        pk.sample_tokens(logits, noise, mask=torch.ones((4, 4), dtype=torch.int64, device=cuda_device))
    with pytest.raises(ValueError):
        pk.sample_tokens(logits, noise, mask=torch.ones((4, 3), dtype=torch.int32, device=cuda_device))
    for bad in ({"temperature": -0.5}, {"temperature": float("nan")}, {"top_p": float("nan")}, {"min_p": float("nan")}):
        with pytest.raises(pk.ProfkError) as e:
            pk.sample_tokens(logits, noise, **bad)
        assert e.value.code == -1
    with pytest.raises(pk.ProfkError):
        pk.sample_tokens(logits[:1].expand(4, 100), noise)  # rows of logits may not overlap
    with pytest.raises(ValueError):
        pk.sample_tokens(logits, noise, out=(torch.empty(3, dtype=torch.int64, device=cuda_device),
                                             torch.empty(4, device=cuda_device)))
