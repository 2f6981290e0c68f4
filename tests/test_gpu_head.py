"""Log-probabilities of given tokens from hidden states and the output matrix."""
import numpy as np
import pytest
import torch

from oracle import logprobs as ref
from logprob_checks import as_numpy, close, row_error, sizes

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


def inputs(rows, width, n, dtype, *, pad=0, seed=0, left_out=0.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed + n)
    ld = -(-width // 8) * 8 + pad
    # (The padding is no part of the product, whatever it holds.)
    def matrix(count, scale):
        m = torch.full((count, ld), float("nan"), device=device, dtype=dtype)
        m[:, :width] = (torch.randn((count, width), generator=g, device=device) * scale).to(dtype)
        return m[:, :width]
    hidden, weight = matrix(rows, 1.0), matrix(n, 2.0 * width ** -0.5)
    tokens = torch.randint(n, (rows,), generator=g, device=device)
    if left_out:
        tokens = torch.where(torch.rand(rows, generator=g, device=device) < left_out, -1, tokens)
    return hidden, weight, tokens


def check(pk, hidden, weight, tokens, T=1.0, **how):
    # The products are exact in float32; their sums are taken sixteen at a time, each step off by at most 2^-23 of
    # the terms' sizes (a sum that is cut off, not rounded), and so is each of the sixteen when they are lined up.
    h, w = as_numpy(hidden), as_numpy(weight)
    z, size = h @ w.T, np.abs(h) @ np.abs(w).T
    t, T64 = tokens.cpu().numpy(), as_numpy(T) if isinstance(T, torch.Tensor) else T
    lp, H = ref.logprobs(z, t, T64)
    x, mean = sizes(z, T64)
    off = (h.shape[1] / 16 + 32) * 2.0 ** -23 * size.max(1) / T64
    at = np.take_along_axis(x, np.clip(t, 0, len(w) - 1)[:, None], 1)[:, 0]
    live = t >= 0
    r = pk.token_logprobs(hidden, tokens, weight=weight, temperature=T, entropy=True, **how)
    close(as_numpy(r.logprobs), lp, np.where(live, 2 * off + row_error(mean, at, lp), 0), "logprobs")
    # d H / d z_i = -p_i (log p_i + H): the sizes of log p_i + H under p are the mean of x and H.
    close(as_numpy(r.entropies), H, np.where(live, off * (2 * mean + 2 * np.abs(H)) + row_error(mean, value=H) + 2.0 ** -18 * mean, 0), "entropies")
    without = pk.token_logprobs(hidden, tokens, weight=weight, temperature=T, **how)
    close(as_numpy(without.logprobs), lp, np.where(live, 2 * off + row_error(mean, at, lp), 0), "logprobs alone")
    assert without.entropies is None and r.stats is None
    return r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,n", [(1, 1, 1), (1, 8, 3), (3, 17, 40), (5, 64, 255), (17, 65, 256), (2, 100, 257), (129, 72, 513),
                                          (128, 128, 512), (64, 1000, 1000), (300, 333, 1500), (1, 1024, 5001), (16, 512, 40000),
                                          (7, 2048, 3001), (257, 40, 20011), (1000, 16, 700), (130, 2049, 700), (64, 4100, 600),
                                          (3, 9000, 300), (300, 2112, 40000)])
def test_sizes(pk, cuda_device, dtype, rows, width, n):
    hidden, weight, tokens = inputs(rows, width, n, dtype, left_out=0.2)
    tokens[0], tokens[-1] = 0, n - 1
    check(pk, hidden, weight, tokens)
    hidden, weight, tokens = inputs(rows, width, n, dtype, pad=8, seed=1)
    check(pk, hidden, weight, tokens, 0.7)


def test_many_tiles(pk, cuda_device):
    # More tiles than the SMs take at once, in both directions.
    for rows, width, n in ((700, 64, 30011), (2500, 24, 9000)):
        hidden, weight, tokens = inputs(rows, width, n, torch.bfloat16)
        check(pk, hidden, weight, tokens)


def test_temperatures_and_left_out_rows(pk, cuda_device):
    hidden, weight, tokens = inputs(150, 96, 1001, torch.bfloat16, left_out=0.3)
    T = 0.3 + torch.rand(150, device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(1))
    r = check(pk, hidden, weight, tokens, T)
    hidden = hidden.clone()
    hidden[tokens < 0] = float("nan")
    again = pk.token_logprobs(hidden, tokens, weight=weight, temperature=T, entropy=True)
    assert torch.equal(again.logprobs, r.logprobs) and torch.equal(again.entropies, r.entropies)
    live = torch.nonzero(tokens >= 0)[:3, 0]
    T[live[0]], tokens[live[1]] = 0.0, 1001
    hidden[live[2], 5] = float("inf")
    again = pk.token_logprobs(hidden, tokens, weight=weight, temperature=T)
    assert again.logprobs[live].isnan().all()
    rest = torch.ones(150, dtype=torch.bool, device=cuda_device)
    rest[live] = False
    assert torch.equal(again.logprobs[rest], r.logprobs[rest])


def test_agrees_with_logits(pk, cuda_device):
    # bfloat16 products of small whole numbers are exact: the same logits, by both ways.
    g = torch.Generator(device=cuda_device).manual_seed(2)
    hidden = torch.randint(-3, 4, (70, 40), generator=g, device=cuda_device).bfloat16()
    weight = torch.randint(-3, 4, (900, 40), generator=g, device=cuda_device).bfloat16()
    tokens = torch.randint(900, (70,), generator=g, device=cuda_device)
    a = pk.token_logprobs(hidden, tokens, weight=weight, temperature=20.0, entropy=True)
    b = pk.token_logprobs(hidden.float() @ weight.float().t(), tokens, temperature=20.0, entropy=True)
    close(as_numpy(a.logprobs), as_numpy(b.logprobs), 2.0 ** -16)
    close(as_numpy(a.entropies), as_numpy(b.entropies), 2.0 ** -16)


def test_no_rows_and_refusals(pk, cuda_device):
    hidden, weight, tokens = inputs(10, 64, 100, torch.bfloat16)
    assert pk.token_logprobs(hidden[:0], tokens[:0], weight=weight).logprobs.shape == (0,)
    r = pk.token_logprobs(hidden, tokens, weight=weight)
    odd = torch.zeros((100, 65), dtype=torch.bfloat16, device=cuda_device)
    for call, error, words in (
            (lambda: pk.token_logprobs(hidden.float(), tokens, weight=weight.float()), TypeError, "bfloat16 or float16"),
            (lambda: pk.token_logprobs(hidden, tokens, weight=weight.half()), TypeError, "weight must be a BFloat16"),
            (lambda: pk.token_logprobs(hidden, tokens, weight=weight[:, :63]), ValueError, r"weight must have shape \(100, 64\)"),
            (lambda: pk.token_logprobs(hidden, tokens, weight=weight.t()), ValueError, "shape"),
            (lambda: pk.token_logprobs(hidden, tokens, weight=weight[0]), ValueError, "2-D"),
            (lambda: pk.token_logprobs(hidden, tokens, weight=odd[:, :64]), ValueError, "16-byte"),
            (lambda: pk.token_logprobs(hidden, tokens, weight=odd[:, 1:]), ValueError, "16-byte"),
            (lambda: pk.token_logprobs(hidden, tokens, weight=weight[:0]), ValueError, "empty"),
            (lambda: pk.token_logprobs(hidden.requires_grad_(), tokens, weight=weight), ValueError, "no gradient"),
            (lambda: pk.token_logprobs(hidden.detach(), tokens, weight=weight.requires_grad_()), ValueError, "no gradient"),
            (lambda: pk.token_logprobs_backward(hidden, tokens, r), ValueError, "hidden states")):
        with pytest.raises(error, match=words):
            call()
    with torch.no_grad():
        assert torch.equal(pk.token_logprobs(hidden, tokens, weight=weight).logprobs, r.logprobs)


@pytest.mark.parametrize("width", [1000, 2048, 3000, 6000])
def test_deep_products_keep_their_precision(pk, cuda_device, width):
    # The tensor cores cut sums off: each of the 128 steps of a segment of 2048 products loses half a unit of the sum so
    # far on average (2^-24), and that is half of the whole on average: 128 * 2^-24 / 2 = 2^-18 of a logit; a
    # log-probability is the difference of two such, of no more than its own size and twice it.  (One segment of 6000
    # would be 2^-16.4.)
    hidden, weight, tokens = inputs(500, width, 700, torch.float16)
    got = as_numpy(pk.token_logprobs(hidden, tokens, weight=weight).logprobs)
    want, _ = ref.logprobs(as_numpy(hidden) @ as_numpy(weight).T, tokens.cpu().numpy())
    assert np.linalg.norm(got - want) < 2.0 ** -18 * np.linalg.norm(want)


@pytest.mark.parametrize("T", [0.3, 0.6, 1.0])
def test_entropies_at_low_temperatures(pk, cuda_device, T):
    # As above, with 1 / T of it and segments the shorter for that: the same bound, twice for an entropy's own sum.
    hidden, weight, tokens = inputs(400, 1502, 900, torch.float16)
    got = pk.token_logprobs(hidden, tokens, weight=weight, temperature=T, entropy=True)
    z = as_numpy(hidden) @ as_numpy(weight).T
    lp, H = ref.logprobs(z, tokens.cpu().numpy(), T)
    assert np.linalg.norm(as_numpy(got.logprobs) - lp) < 2.0 ** -18 * np.linalg.norm(lp)
    assert np.linalg.norm(as_numpy(got.entropies) - H) < 2.0 ** -17 * np.linalg.norm(np.maximum(H, 1))
    per_row = torch.full((400,), T, device=cuda_device)
    again = pk.token_logprobs(hidden, tokens, weight=weight, temperature=per_row, entropy=True)
    assert np.linalg.norm(as_numpy(again.entropies) - H) < 2.0 ** -17 * np.linalg.norm(np.maximum(H, 1))


@pytest.mark.parametrize("width", [200, 2500])
def test_a_wait_that_runs_out(pk, cuda_device, width):
    # A barrier that waits for one arrival more than comes, with a bound of 4096 polls: the kernel gives up and says so.
    hidden, weight, tokens = inputs(300, width, 9000, torch.bfloat16)
    tokens[5] = -1
    want = pk.token_logprobs(hidden, tokens, weight=weight)
    pk.set_option(pk.OPT_HEAD_WAIT_TEST, 1)
    got = pk.token_logprobs(hidden, tokens, weight=weight, entropy=True)
    torch.cuda.synchronize()
    pk.set_option(pk.OPT_HEAD_WAIT_TEST, 0)
    live = tokens >= 0
    assert got.logprobs[live].isnan().all() and got.entropies[live].isnan().all() and got.logprobs[5] == 0
    assert torch.equal(pk.token_logprobs(hidden, tokens, weight=weight).logprobs, want.logprobs)


def test_streams_graphs_and_equal_bits(pk, cuda_device):
    hidden, weight, tokens = inputs(200, 512, 5000, torch.bfloat16)
    want = pk.token_logprobs(hidden, tokens, weight=weight, entropy=True)
    for _ in range(3):
        again = pk.token_logprobs(hidden, tokens, weight=weight, entropy=True)
        assert torch.equal(again.logprobs, want.logprobs) and torch.equal(again.entropies, want.entropies)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = pk.token_logprobs(hidden, tokens, weight=weight, stream=side)
    side.synchronize()
    assert torch.equal(got.logprobs, want.logprobs)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(pk.token_logprobs(hidden, tokens, weight=weight))
    hidden.copy_(hidden.flip(0))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for stream, graph in zip(streams, graphs):  # two captured calls side by side
        with torch.cuda.stream(stream):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    want = pk.token_logprobs(hidden, tokens, weight=weight)
    assert all(torch.equal(out.logprobs, want.logprobs) for out in outs)
