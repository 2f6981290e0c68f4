"""Log-probabilities of given tokens, from logits: values, entropies, gradients, and what the calls refuse."""
import numpy as np
import pytest
import torch

from oracle import logprobs as ref
from logprob_checks import as_numpy, close, gradient_error, make, row_error, sizes

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


def check(pk, logits, tokens, T=1.0, seed=3, out=None, entropy=True):
    rows, n = logits.shape
    l, t, T64 = as_numpy(logits), tokens.cpu().numpy(), as_numpy(T) if isinstance(T, torch.Tensor) else T
    lp, H = ref.logprobs(l, t, T64)
    x, mean = sizes(l, T64)
    at = np.take_along_axis(x, np.clip(t, 0, n - 1)[:, None], 1)[:, 0] if rows else np.zeros(0)
    r = pk.token_logprobs(logits, tokens, temperature=T, entropy=entropy)
    close(as_numpy(r.logprobs), lp, row_error(mean, at, lp), "logprobs")
    if entropy:
        close(as_numpy(r.entropies), H, row_error(mean, value=H) + 2.0 ** -18 * mean, "entropies")
    g = torch.Generator(device=logits.device).manual_seed(seed)
    dg = torch.randn(rows, generator=g, device=logits.device)
    dh = torch.randn(rows, generator=g, device=logits.device) if entropy else None
    want = ref.gradient(l, t, T64, as_numpy(dg), as_numpy(dh) if entropy else None)
    got = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=dg, grad_entropies=dh, out=out)
    assert got.dtype == logits.dtype and got.shape == logits.shape
    close(as_numpy(got), want, gradient_error(l, T64, as_numpy(dg), as_numpy(dh) if entropy else None, want, logits.dtype), "gradient")
    return r, got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n,ld,offset", [(1, 1, 0, 0), (3, 2, 5, 1), (7, 9, 0, 0), (33, 64, 64, 3), (9, 513, 0, 0), (5, 2048, 2056, 0),
                                              (4, 4095, 4097, 1), (3, 5000, 0, 2), (2, 8192, 0, 0), (1, 32768, 0, 0), (3, 40001, 0, 0),
                                              (170, 6001, 0, 0), (320, 4500, 4504, 0)])
def test_sizes_and_strides(pk, cuda_device, dtype, rows, n, ld, offset):
    logits, tokens, _ = make(rows, n, dtype, ld, offset=offset, left_out=0.2)
    tokens[0], tokens[-1] = 0, n - 1  # the first and the last of a row
    for entropy in (True, False):
        check(pk, logits, tokens, entropy=entropy)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [0.05, 0.7, 1.0, 30.0])
def test_temperatures(pk, cuda_device, dtype, T):
    logits, tokens, g = make(11, 4999, dtype)
    a, da = check(pk, logits, tokens, T)
    per_row = torch.full((11,), T, device=cuda_device)
    b, db = check(pk, logits, tokens, per_row)
    assert torch.equal(a.logprobs, b.logprobs) and torch.equal(da, db)
    check(pk, logits, tokens, per_row * (0.5 + torch.rand(11, generator=g, device=cuda_device)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [40, 5003])
def test_rows_at_their_limits(pk, cuda_device, dtype, n):
    logits, tokens, _ = make(12, n, dtype)
    lowest = torch.finfo(dtype).min
    logits[0] = -INF                       # nothing at all
    logits[1, 1:] = -INF                   # one token, and the row asks for another or for it
    logits[2, 1:] = -INF
    tokens[1], tokens[2] = 0, n - 1
    logits[3] = lowest                     # masks of the type's lowest value: an even row
    logits[4, : n // 2] = lowest
    logits[5, 3] = float("nan")
    logits[6, n - 1] = INF
    logits[7] = float("nan")               # left out: what it holds does not matter
    tokens[7] = -1
    logits[8] = torch.finfo(dtype).max
    logits[9, :] = 0
    logits[10] = -INF
    logits[10, n - 2] = lowest
    tokens[10] = n - 2
    tokens[11] = n                         # no such token
    check(pk, logits, tokens)
    r = pk.token_logprobs(logits, tokens, entropy=True)
    lp, H = r.logprobs.tolist(), r.entropies.tolist()
    assert lp[0] == -INF and H[0] == 0 and lp[1] == 0 and lp[2] == -INF and H[2] == 0 and lp[10] == 0
    assert all(v != v for v in (lp[5], lp[6], lp[11])) and lp[7] == 0 and H[7] == 0
    one = torch.ones(12, device=cuda_device)
    grad = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=one).float()
    assert (grad[0] == 0).all() and (grad[7] == 0).all() and grad[5].isnan().all() and grad[11].isnan().all()
    zero = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=0 * one, grad_entropies=0 * one)
    assert (zero == 0).all()  # the NaN rows too: nothing is asked of them
    assert (pk.token_logprobs_backward(logits, tokens, r) == 0).all()


@pytest.mark.parametrize("n", [50, 301, 6001])
@pytest.mark.parametrize("base", [3e2, 3e5, 7e5, 1e6, 1e9, -7e5, -1e9])
def test_logits_far_from_zero(pk, cuda_device, n, base):
    # Only differences count; single elements at a row's ends and whole vectors have to agree on what they are taken from.
    logits, tokens, _ = make(9, n, torch.float32, n + 1, offset=3)
    logits += base
    for r in range(9):  # the largest one at the ends, and next to them
        logits[r, r if r < 5 else n - 10 + r] += 2 * abs(base) * 2.0 ** -23 + 4
    check(pk, logits, tokens)
    check(pk, logits, tokens, 0.01 if abs(base) > 1e8 else 0.3)


def test_a_rows_own_bad_temperature(pk, cuda_device):
    for n in (64, 6000):
        logits, tokens, _ = make(5, n, torch.float32)
        T = torch.tensor([1.0, 0.0, -1.0, float("nan"), INF], device=cuda_device)
        r = pk.token_logprobs(logits, tokens, temperature=T, entropy=True)
        good = pk.token_logprobs(logits[:1], tokens[:1])
        assert torch.equal(r.logprobs[:1], good.logprobs) and r.logprobs[1:].isnan().all()
        grad = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=torch.ones(5, device=cuda_device))
        assert grad[1:].isnan().all() and not grad[0].isnan().any()


@pytest.mark.parametrize("dtype", TYPES)
def test_no_rows(pk, cuda_device, dtype):
    logits = torch.empty((0, 100), dtype=dtype, device=cuda_device)
    tokens = torch.empty(0, dtype=torch.int64, device=cuda_device)
    r = pk.token_logprobs(logits, tokens, entropy=True)
    assert r.logprobs.shape == (0,) and pk.token_logprobs_backward(logits, tokens, r).shape == (0, 100)


def test_sampled_tokens_have_their_log_probabilities(pk, cuda_device):
    logits, _, g = make(40, 3001, torch.bfloat16)
    logits[:, 2990:] = -INF
    noise = torch.empty((40, 3001), device=cuda_device).exponential_(generator=g)
    tokens, lp = pk.sample_tokens(logits, noise, temperature=0.8)
    again = pk.token_logprobs(logits, tokens, temperature=0.8).logprobs
    # Both are off the exact value by row_error at most, and sample_tokens' weights are rounded to 2^-24 of the largest.
    _, mean = sizes(as_numpy(logits), 0.8)
    close(as_numpy(again), as_numpy(lp), 2 * row_error(mean, as_numpy(lp), as_numpy(lp)) + 3001 * 2.0 ** -24)


@pytest.mark.parametrize("n,ld", [(300, 300), (6000, 6008)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_to_a_given_place(pk, cuda_device, dtype, n, ld):
    logits, tokens, _ = make(6, n, dtype, ld, left_out=0.3)
    r, want = check(pk, logits, tokens)
    dg = torch.randn(6, device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(3))
    dh = torch.randn(6, device=cuda_device, generator=(g := torch.Generator(device=cuda_device).manual_seed(3)))
    dh = torch.randn(6, device=cuda_device, generator=g)
    for shift in range(0, 9):  # another alignment than the logits', and an odd row stride
        store = torch.full((6 * (n + 5) + 9,), 7.0, dtype=dtype, device=cuda_device)
        out = store[shift:shift + 6 * (n + 5)].view(6, n + 5)[:, :n]
        got = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=dg, grad_entropies=dh, out=out)
        assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)
        out.fill_(7.0)
        assert (store == 7).all()  # nothing beside it was written
    place = logits.clone() if ld == n else torch.empty((6, ld), dtype=dtype, device=cuda_device)[:, :n].copy_(logits)
    assert torch.equal(pk.token_logprobs_backward(place, tokens, r, grad_logprobs=dg, grad_entropies=dh, out=place), want)
    with pytest.raises(pk.ProfkError):  # across the logits
        both = torch.zeros(12, n, dtype=dtype, device=cuda_device)
        pk.token_logprobs_backward(both[:6], tokens, r, grad_logprobs=dg, out=both[1:7])
    with pytest.raises(ValueError):
        pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=dg, out=torch.empty(n, dtype=dtype, device=cuda_device).expand(6, n))


@pytest.mark.parametrize("n", [50, 9000])
def test_autograd(pk, cuda_device, n):
    logits, tokens, g = make(9, n, torch.float32, left_out=0.2)
    a, b = torch.randn(9, generator=g, device=cuda_device), torch.randn(9, generator=g, device=cuda_device)
    leaf = logits.clone().requires_grad_()
    r = pk.token_logprobs(leaf, tokens, temperature=0.9, entropy=True)
    assert r.logprobs.requires_grad and r.entropies.requires_grad and not r.stats.requires_grad
    ((r.logprobs * a).sum() + (r.entropies * b).sum()).backward()
    want = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=a, grad_entropies=b)
    assert torch.equal(leaf.grad, want)
    leaf.grad = None
    pk.token_logprobs(leaf, tokens).logprobs.sum().backward()  # an expanded gradient
    live = (tokens >= 0).float()
    close(as_numpy(leaf.grad.sum(1)), 0 * as_numpy(live), 2.0 ** -15)
    with torch.no_grad():
        assert not pk.token_logprobs(leaf, tokens).logprobs.requires_grad
    bf = logits.bfloat16().requires_grad_()
    pk.token_logprobs(bf, tokens).logprobs.mean().backward()
    assert bf.grad.dtype == torch.bfloat16
    with pytest.raises(ValueError, match="current stream"):
        pk.token_logprobs(leaf, tokens, stream=torch.cuda.Stream())
    with pytest.raises(ValueError, match="constant"):
        pk.token_logprobs(leaf, tokens, temperature=torch.ones(9, device=cuda_device, requires_grad=True))


def test_gradient_against_differences(pk, cuda_device):
    # Central differences of the library's own float32 values: h = 2^-4 leaves h^2 / 6 times third derivatives (at most 1
    # for each of two terms) and 2 row_error / 2h of rounding.
    logits, tokens, g = make(6, 30, torch.float32, spread=1.0)
    a, b = torch.randn(6, generator=g, device=cuda_device), torch.randn(6, generator=g, device=cuda_device)
    r = pk.token_logprobs(logits, tokens, temperature=1.0, entropy=True)
    grad = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=a, grad_entropies=b)
    h = 2.0 ** -4

    def value(l):
        r = pk.token_logprobs(l, tokens, entropy=True)
        return (r.logprobs * a + r.entropies * b).double()
    scale = a.abs() + 6 * b.abs()
    for i in range(30):
        up, down = logits.clone(), logits.clone()
        up[:, i] += h
        down[:, i] -= h
        slope = (value(up) - value(down)) / (up[:, i].double() - down[:, i].double())
        close(as_numpy(slope), as_numpy(grad[:, i]), as_numpy(scale) * (h * h / 6 + 2 * 2.0 ** -17 / (2 * h)))


@pytest.mark.parametrize("rows,n", [(1, 1 << 22), (2, 3_000_001)])
def test_long_rows(pk, cuda_device, rows, n):
    logits, tokens, _ = make(rows, n, torch.bfloat16)
    check(pk, logits, tokens)
    even = torch.zeros((1, 1 << 26), dtype=torch.bfloat16, device=cuda_device)  # every weight the same: 2^26 equal terms
    r = pk.token_logprobs(even, torch.zeros(1, dtype=torch.int64, device=cuda_device), entropy=True)
    want = 26 * np.log(2.0)
    assert abs(r.logprobs.item() + want) < 2.0 ** -18 and abs(r.entropies.item() - want) < 2.0 ** -18


def test_far_offsets(pk, cuda_device):
    # Rows whose elements lie beyond 2^32 bytes and 2^31 elements.
    n, ld = 5000, 1 << 30
    store = torch.empty(3 * ld, dtype=torch.bfloat16, device=cuda_device)
    logits = store.view(3, ld)[:, :n]
    small, tokens, _ = make(3, n, torch.bfloat16)
    logits.copy_(small)
    r = pk.token_logprobs(logits, tokens, entropy=True)
    want = pk.token_logprobs(small, tokens, entropy=True)
    assert torch.equal(r.logprobs, want.logprobs) and torch.equal(r.entropies, want.entropies)
    dg = torch.ones(3, device=cuda_device)
    got = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=dg, out=logits)
    assert torch.equal(got, pk.token_logprobs_backward(small, tokens, want, grad_logprobs=dg))


def test_equal_calls_give_equal_bits(pk, cuda_device):
    for rows, n in ((3, 70000), (400, 300), (200, 9001)):
        logits, tokens, _ = make(rows, n, torch.float16)
        first = pk.token_logprobs(logits, tokens, entropy=True)
        for _ in range(5):
            r = pk.token_logprobs(logits, tokens, entropy=True)
            assert all(torch.equal(x, y) for x, y in zip(first[:3], r[:3]))


@pytest.mark.parametrize("n", [200, 20000])
def test_streams_and_graphs(pk, cuda_device, n):
    logits, tokens, g = make(20, n, torch.bfloat16)
    dg = torch.randn(20, generator=g, device=cuda_device)
    want = pk.token_logprobs(logits, tokens, entropy=True)
    want_grad = pk.token_logprobs_backward(logits, tokens, want, grad_logprobs=dg)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r = pk.token_logprobs(logits, tokens, entropy=True, stream=side)
    grad = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=dg, stream=side)
    side.synchronize()
    assert torch.equal(r.logprobs, want.logprobs) and torch.equal(grad, want_grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = pk.token_logprobs(logits, tokens, entropy=True)
        grad = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=dg)
    logits.copy_(logits.flip(0))
    graph.replay()
    again = pk.token_logprobs(logits, tokens, entropy=True)
    assert torch.equal(r.logprobs, again.logprobs)
    assert torch.equal(grad, pk.token_logprobs_backward(logits, tokens, again, grad_logprobs=dg))


def test_messages(pk, cuda_device):
    z, t, _ = make(10, 16, torch.float32)
    r = pk.token_logprobs(z, t)
    one = torch.ones(10, device=cuda_device)
    for call, error, words in (
            (lambda: pk.token_logprobs(z.double(), t), TypeError, "float32, bfloat16 or float16"),
            (lambda: pk.token_logprobs(z.cpu(), t), TypeError, "CUDA"),
            (lambda: pk.token_logprobs(z[0], t), ValueError, "2-D"),
            (lambda: pk.token_logprobs(z.t(), t), ValueError, "column stride"),
            (lambda: pk.token_logprobs(z, t.int()), TypeError, "tokens must be a Long"),
            (lambda: pk.token_logprobs(z, t[:5]), ValueError, r"tokens must have shape \(10,\), not \(5,\)"),
            (lambda: pk.token_logprobs(z, t, temperature=0.0), ValueError, "temperature"),
            (lambda: pk.token_logprobs(z, t, temperature=float("nan")), ValueError, "temperature"),
            (lambda: pk.token_logprobs(z, t, temperature=1e-45), ValueError, "temperature"),
            (lambda: pk.token_logprobs(z, t, temperature=one[:3]), ValueError, r"temperature must have shape"),
            (lambda: pk.token_logprobs_backward(z, t, r, grad_logprobs=one[:2]), ValueError, "grad_logprobs must have shape"),
            (lambda: pk.token_logprobs_backward(z, t, r, grad_entropies=one), ValueError, "entropy=True"),
            (lambda: pk.token_logprobs_backward(z, t, r, grad_logprobs=one.double()), TypeError, "grad_logprobs must be a Float"),
            (lambda: pk.token_logprobs_backward(z, t, r, grad_logprobs=one, out=z.half()), TypeError, "out must be"),
            (lambda: pk.token_logprobs_backward(z[:5], t[:5], r, grad_logprobs=one), ValueError, "stats must have shape")):
        with pytest.raises(error, match=words):
            call()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", [(5000, 700), (2500, 6000), (4000, 9000), (700, 5000), (1300, 16400), (40, 70001), (5, 300_000)])
def test_many_rows_and_parts(pk, cuda_device, dtype, rows, n):
    # Rows by warps that go on to others, by CTAs, and by clusters of 2 to 8 of them.
    logits, tokens, g = make(rows, n, dtype, left_out=0.1)
    r = pk.token_logprobs(logits, tokens, entropy=True)
    dg = torch.randn(rows, generator=g, device=cuda_device)
    grad = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=dg)
    some = torch.tensor(sorted({0, 1, rows // 2, rows - 2, rows - 1}), device=cuda_device)  # against the definition
    l, t = as_numpy(logits[some]), tokens[some].cpu().numpy()
    lp, H = ref.logprobs(l, t)
    x, mean = sizes(l, 1.0)
    at = np.take_along_axis(x, np.clip(t, 0, n - 1)[:, None], 1)[:, 0]
    close(as_numpy(r.logprobs[some]), lp, row_error(mean, at, lp))
    close(as_numpy(r.entropies[some]), H, row_error(mean, value=H) + 2.0 ** -18 * mean)
    want = ref.gradient(l, t, 1.0, as_numpy(dg[some]))
    close(as_numpy(grad[some]), want, gradient_error(l, 1.0, as_numpy(dg[some]), None, want, dtype))
    # and all of them against the same rows in smaller batches, which go other ways through the kernels
    for part in torch.arange(rows, device=cuda_device).split(max(1, rows // 7)):
        q = pk.token_logprobs(logits[part], tokens[part], entropy=True)
        torch.testing.assert_close(q.logprobs, r.logprobs[part], rtol=2.0 ** -20, atol=2.0 ** -17)
        torch.testing.assert_close(q.entropies, r.entropies[part], rtol=2.0 ** -20, atol=2.0 ** -16)


def test_host_threads(pk, cuda_device):
    # Four threads, each with inputs and a stream of its own.
    import threading

    def work(i, out):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            n = (200, 3000, 40000, 9000)[i]
            logits, tokens, g = make(20 + i, n, torch.bfloat16, seed=i)
            zero = torch.zeros(20 + i, device=cuda_device)
            for _ in range(30):
                r = pk.token_logprobs(logits, tokens, entropy=True)
                p = pk.policy_loss(logits, tokens, r.logprobs, 1 + zero, gradient=True)
                d = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=1 + zero)
                h = pk.token_logprobs(logits[:, :184], tokens % 64, weight=logits[:8, :184].contiguous().repeat(8, 1)) if n % 8 == 0 else r
            stream.synchronize()
            out[i] = [t.cpu() for t in (r.logprobs, r.entropies, p.loss, p.grad_logits, d, h.logprobs)]

    alone, together = {}, {}
    for i in range(4):
        work(i, alone)
    threads = [threading.Thread(target=work, args=(i, together)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(a, b) for i in range(4) for a, b in zip(alone[i], together[i]))


@pytest.mark.parametrize("call", ["logprobs", "backward", "policy", "preference", "head"])
def test_outputs_on_another_stream_leave_freed_blocks_alone(pk, cuda_device, call):
    # Work queued on the current stream on tensors that have been let go: outputs of a call on another stream must not
    # be made from their memory.
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        z, t, g = make(512, 640, torch.bfloat16)
        one = torch.ones(512, device=cuda_device)
        o = torch.arange(0, 513, 64, device=cuda_device)
        r = pk.token_logprobs(z, t, entropy=True)
        few = t % 64
    calls = {"logprobs": lambda **s: pk.token_logprobs(z, t, entropy=True, **s)[:3],
             "backward": lambda **s: (pk.token_logprobs_backward(z, t, r, grad_logprobs=one, **s),),
             "policy": lambda **s: [v for v in pk.policy_loss(z, t, r.logprobs, one, gradient=True, **s)[:10] if v is not None],
             "preference": lambda **s: pk.preference_loss(z, t, o[:5], **s)[:5],
             "head": lambda **s: pk.token_logprobs(z, few, weight=z[:64], entropy=True, **s)[:2]}
    with torch.cuda.stream(side):
        want = calls[call]()
    torch.cuda.synchronize()
    freed = [torch.full((v.untyped_storage().nbytes() // 4,), 7.0, device=cuda_device) for v in want]
    kept = [torch.zeros_like(f) for f in freed]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    for a, b in zip(kept, freed):
        a.copy_(b)
    spans = [(f.data_ptr(), f.data_ptr() + f.numel() * 4) for f in freed]
    del freed, a, b
    got = calls[call](stream=side)
    assert not any(lo <= v.data_ptr() < hi for v in got for lo, hi in spans)
    side.synchronize()
    assert all(torch.equal(x.cpu(), y.cpu()) for x, y in zip(got, want))
    torch.cuda.synchronize()
    assert all((k == 7).all() for k in kept)


def test_forward_mode_and_transforms_are_refused(pk, cuda_device):
    import torch.autograd.forward_ad as fwd
    z, t, _ = make(10, 16, torch.float32)
    one = torch.ones(10, device=cuda_device)
    o = torch.tensor([0, 5, 10], device=cuda_device)
    r = pk.token_logprobs(z, t)
    h = z.bfloat16()
    with fwd.dual_level():
        dual = lambda v: fwd.make_dual(v, torch.ones_like(v))  # noqa: E731
        for call in (lambda: pk.token_logprobs(dual(z), t), lambda: pk.token_logprobs(z, t, temperature=dual(one)),
                     lambda: pk.token_logprobs_backward(z, t, r, grad_logprobs=dual(one)), lambda: pk.policy_loss(dual(z), t, one, one),
                     lambda: pk.policy_loss(z, t, dual(one), one), lambda: pk.policy_loss(z, t, one, one, weights=dual(one)),
                     lambda: pk.preference_loss(dual(z), t, o), lambda: pk.preference_loss(z, t, o, ref_logprobs=dual(one)),
                     lambda: pk.token_logprobs(dual(h), t, weight=h), lambda: pk.token_logprobs(h, t, weight=dual(h))):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
    with pytest.raises(Exception):
        torch.func.grad(lambda v: pk.token_logprobs(v, t).logprobs.sum())(z)
    with pytest.raises(Exception):
        torch.vmap(lambda v: pk.token_logprobs(v, t).logprobs)(z.expand(3, 10, 16))


@pytest.mark.parametrize("of", ["logprobs", "policy", "preference"])
def test_a_second_derivative_raises(pk, cuda_device, of):
    z, t, _ = make(10, 16, torch.float32)
    z = z.clone().requires_grad_()
    one = torch.ones(10, device=cuda_device)
    y = {"logprobs": lambda: pk.token_logprobs(z, t).logprobs.sum(), "policy": lambda: pk.policy_loss(z, t, -2 * one, one).loss,
         "preference": lambda: pk.preference_loss(z, t, torch.tensor([0, 5, 10], device=cuda_device)).loss}[of]()
    grad, = torch.autograd.grad(y, z, create_graph=True)
    with pytest.raises(NotImplementedError):
        (y * 0 + grad.square().sum()).backward()


def test_inputs_changed_in_between_are_noticed(pk, cuda_device):
    z, t, _ = make(10, 16, torch.float32)
    z = z.clone().requires_grad_()
    for change in ("logits", "tokens"):
        x = z * 1.0
        tokens = t.clone()
        r = pk.token_logprobs(x, tokens)
        (x.detach() if change == "logits" else tokens).zero_()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            r.logprobs.sum().backward()
