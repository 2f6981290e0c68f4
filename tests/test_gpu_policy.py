"""The clipped policy loss and the preference loss: values, slopes, gradients, what leaves a token out."""
import numpy as np
import pytest
import torch

from oracle import logprobs as ref
from logprob_checks import as_numpy, close, gradient_error, make, row_error, sizes

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


def policy_inputs(rows, n, dtype, *, ld=0, T=1.0, seed=0, left_out=0.0, offset=0):
    logits, tokens, g = make(rows, n, dtype, ld, seed=seed, left_out=left_out, offset=offset)
    lp, H = ref.logprobs(as_numpy(logits), tokens.cpu().numpy(), T)
    dev = logits.device
    # Ratios well away from the clips' borders: 0.5 .. 0.75, 0.85 .. 1.15, 1.35 .. 2.
    ratio = torch.where(torch.rand(rows, generator=g, device=dev) < 0.5, 0.85 + 0.3 * torch.rand(rows, generator=g, device=dev),
                        torch.where(torch.rand(rows, generator=g, device=dev) < 0.5, 0.5 + 0.25 * torch.rand(rows, generator=g, device=dev),
                                    1.35 + 0.65 * torch.rand(rows, generator=g, device=dev)))
    now = torch.from_numpy(lp).to(dev)
    old = (now - ratio.double().log()).float()
    refs = (now + 0.3 * torch.randn(rows, generator=g, device=dev)).float()
    A = torch.randn(rows, generator=g, device=dev)
    w = torch.rand(rows, generator=g, device=dev) / rows
    if rows > 4:
        w[rows // 2] = 0
        A[rows // 3] = 0
    return logits, tokens, old, A, refs, w, lp, H


def check_policy(pk, rows, n, dtype, *, ld=0, T=1.0, kl=0.1, entropy=0.05, with_ref=True, weights=True, left_out=0.0, low=0.2, high=0.28, out=None, offset=0):
    logits, tokens, old, A, refs, w, lp, H = policy_inputs(rows, n, dtype, ld=ld, T=T, left_out=left_out, offset=offset)
    refs, w = (refs if with_ref else None), (w if weights else None)
    l, t = as_numpy(logits), tokens.cpu().numpy()
    w64 = as_numpy(w) if weights else np.full(rows, 1.0 / rows)
    live = (t >= 0) & (w64 != 0)
    want = ref.policy(lp, H, as_numpy(old), as_numpy(A), None if refs is None else as_numpy(refs), w64, live, low, high,
                      kl, entropy or 0.0)
    how = dict(ref_logprobs=refs, weights=w, temperature=T, clip_low=low, clip_high=high, kl=kl, entropy=entropy)
    fused = pk.policy_loss(logits, tokens, old, A, gradient=True, out=out, **how)
    plain = pk.policy_loss(logits, tokens, old, A, **how)
    assert plain.grad_logits is None
    x, mean = sizes(l, T)
    at = np.take_along_axis(x, np.clip(t, 0, n - 1)[:, None], 1)[:, 0]
    d = np.where(live, row_error(mean, at, lp), 0.0)  # of the log-probabilities
    dH = np.where(live, row_error(mean, value=H) + 2.0 ** -18 * mean, 0.0)
    # A term moves with lp by its slopes: A r and kl (e^q - 1), and each of its few operations by a step.
    ratio, A64 = np.exp(lp - as_numpy(old)), np.abs(as_numpy(A))
    e = np.exp(as_numpy(refs) - lp) if with_ref else np.zeros(rows)
    moves = A64 * ratio + abs(kl) * (e + 1)
    step = d + 2.0 ** -22 * (1 + np.abs(as_numpy(old) - lp))
    term = np.where(live, w64 * (moves * step + abs(entropy or 0) * dH), 0.0).sum()
    # A slope is w (-A r + kl (1 - e^q)): relative to lp's error and its own operations.
    ds = np.where(live, w64 * moves * 2 * step, 0.0)
    for r in (fused, plain):  # (not by the same kernel: a row's sums may be added up in another order)
        close(as_numpy(r.logprobs), np.where(live, lp, 0.0), d, "logprobs")
        close(as_numpy(r.loss), want[0], term + 2.0 ** -23 * abs(want[0]), "loss")
        close(as_numpy(r.kl), want[1], np.where(live, w64 * (e + 1) * step, 0).sum(), "kl")
        close(as_numpy(r.clipped), want[2], 2.0 ** -23 * want[2], "clipped")
        if entropy is not None:
            close(as_numpy(r.entropies), np.where(live, H, 0.0), dH, "entropies")
            close(as_numpy(r.entropy), want[3], np.where(live, w64 * dH, 0).sum() + 2.0 ** -23 * want[3], "entropy")
        else:
            assert r.entropies is None and r.entropy == 0
        close(as_numpy(r.slopes), want[4], ds, "slopes")
        if entropy:
            close(as_numpy(r.entropy_slopes), want[5], 2.0 ** -23 * np.abs(want[5]), "entropy slopes")
        else:
            assert r.entropy_slopes is None
    grad = ref.gradient(l, t, T, want[4], want[5])
    off = gradient_error(l, T, want[4], want[5], grad, dtype)
    p = np.where(np.isfinite(l), np.exp(-x), 0.0)
    p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    off = off + (ds / T)[:, None] * (p + (np.arange(n) == t[:, None]))
    got = as_numpy(fused.grad_logits)
    close(got, grad, off, "gradient with the loss")
    back = pk.policy_loss_backward(logits, tokens, plain)
    close(as_numpy(back), grad, off, "gradient after the loss")
    two = torch.full((), 2.0, device=logits.device)
    twice = as_numpy(pk.policy_loss_backward(logits, tokens, plain, grad_loss=two))
    close(twice, 2 * grad, 2 * off, "of twice the loss")
    dead = torch.from_numpy(~live).to(logits.device)
    assert (fused.grad_logits[dead] == 0).all() and (back[dead] == 0).all()
    return fused


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n,ld,offset", [(1, 2, 0, 0), (6, 65, 0, 0), (40, 513, 515, 1), (5, 4100, 0, 0), (1, 32768, 0, 0), (9, 20001, 0, 0),
                                              (7, 20001, 20008, 0), (310, 4600, 0, 0), (600, 150, 0, 0)])
def test_policy_sizes(pk, cuda_device, dtype, rows, n, ld, offset):
    check_policy(pk, rows, n, dtype, ld=ld, offset=offset, left_out=0.2)


@pytest.mark.parametrize("n", [400, 12001])
@pytest.mark.parametrize("how", [dict(with_ref=False), dict(kl=0.0), dict(entropy=None), dict(entropy=0.0), dict(weights=False),
                                 dict(T=0.6), dict(low=0.1, high=0.5), dict(with_ref=False, entropy=None, weights=False), dict(kl=-0.1, entropy=-0.2)])
def test_policy_terms(pk, cuda_device, n, how):
    check_policy(pk, 30, n, torch.bfloat16, left_out=0.2, **how)


def test_policy_of_many_tokens(pk, cuda_device):
    check_policy(pk, 5000, 64, torch.float32, left_out=0.1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [100, 9000])
def test_left_out_tokens_hold_anything(pk, cuda_device, dtype, n):
    logits, tokens, old, A, refs, w, _, _ = policy_inputs(12, n, dtype)
    how = dict(ref_logprobs=refs, kl=0.1, entropy=0.1)
    w[2] = w[5] = 0
    tokens[7] = -1
    want = pk.policy_loss(logits, tokens, old, A, weights=w, gradient=True, **how)
    bad = torch.tensor([2, 5, 7], device=cuda_device)
    logits[bad], old[bad], A[bad], refs[bad] = float("nan"), INF, float("nan"), float("nan")
    got = pk.policy_loss(logits, tokens, old, A, weights=w, gradient=True, **how)
    assert torch.equal(got.loss, want.loss) and torch.equal(got.grad_logits, want.grad_logits) and all(torch.equal(a, b) for a, b in zip(got[:4], want[:4]))
    assert (got.grad_logits[bad] == 0).all() and (got.logprobs[bad] == 0).all()
    back = pk.policy_loss_backward(logits, tokens, got)
    assert (back[bad] == 0).all() and not back.isnan().any()
    # What is not left out shows.
    logits[3, 1] = float("nan")
    got = pk.policy_loss(logits, tokens, old, A, weights=w, gradient=True, **how)
    assert got.loss.isnan() and got.grad_logits[3].isnan().all() and not got.grad_logits[4].isnan().any()


def test_no_token_at_all(pk, cuda_device):
    logits, tokens, old, A, refs, w, _, _ = policy_inputs(12, 5000, torch.bfloat16)
    r = pk.policy_loss(logits, tokens, old, A, weights=0 * w, ref_logprobs=refs, kl=1.0, entropy=1.0, gradient=True)
    assert (r.grad_logits == 0).all() and all(t == 0 for t in r[:4])
    none = torch.empty(0, device=cuda_device)
    r = pk.policy_loss(logits[:0], tokens[:0], none, none, gradient=True)
    assert r.loss == 0 and r.grad_logits.shape == (0, 5000) and r.kl == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [100, 9000, 9001])
def test_gradient_in_the_logits_place(pk, cuda_device, dtype, n):
    logits, tokens, old, A, refs, w, _, _ = policy_inputs(20, n, dtype, left_out=0.2)
    want = pk.policy_loss(logits, tokens, old, A, ref_logprobs=refs, weights=w, kl=0.1, entropy=0.1, gradient=True)
    wide = torch.full((20, n + 3), 7.0, dtype=dtype, device=cuda_device)
    got = pk.policy_loss(logits, tokens, old, A, ref_logprobs=refs, weights=w, kl=0.1, entropy=0.1, gradient=True, out=wide[:, 1:n + 1])
    assert torch.equal(got.grad_logits, want.grad_logits) and (wide[:, 0] == 7).all() and (wide[:, n + 1:] == 7).all()
    place = logits.clone()
    got = pk.policy_loss(place, tokens, old, A, ref_logprobs=refs, weights=w, kl=0.1, entropy=0.1, gradient=True, out=place)
    assert got.grad_logits is place and torch.equal(place, want.grad_logits) and torch.equal(got.loss, want.loss)


@pytest.mark.parametrize("n", [100, 9000])
def test_policy_autograd(pk, cuda_device, n):
    logits, tokens, old, A, refs, w, _, _ = policy_inputs(20, n, torch.float32, left_out=0.2)
    leaf = logits.clone().requires_grad_()
    r = pk.policy_loss(leaf, tokens, old, A, ref_logprobs=refs, weights=w, kl=0.1, entropy=0.1)
    assert r.loss.requires_grad and not r.logprobs.requires_grad and not r.kl.requires_grad and r.grad_logits is None
    (3 * r.loss).backward()
    three = torch.full((), 3.0, device=cuda_device)
    assert torch.equal(leaf.grad, pk.policy_loss_backward(logits, tokens, r, grad_loss=three))
    fused = pk.policy_loss(leaf, tokens, old, A, gradient=True)
    assert not fused.loss.requires_grad
    for name in ("old", "A", "refs", "w"):
        args = dict(old=old, A=A, refs=refs, w=w)
        args[name] = args[name].clone().requires_grad_()
        for l in (leaf, logits):
            with pytest.raises(ValueError, match="constant"):
                pk.policy_loss(l, tokens, args["old"], args["A"], ref_logprobs=args["refs"], weights=args["w"])
        with torch.no_grad():
            pk.policy_loss(leaf, tokens, args["old"], args["A"], ref_logprobs=args["refs"], weights=args["w"])


# ---- preference ----------------------------------------------------------------------------------

def check_preference(pk, lengths, n, dtype, *, ld=0, behind=0, before=0, left_out=0.2, with_ref=True, scale=1.0, spread=1.0, **how):
    rows = before + sum(lengths) + behind
    logits, tokens, g = make(rows, n, dtype, ld, left_out=left_out, spread=spread)
    if behind:
        logits[rows - behind:] = float("nan")  # padding
    if before:
        logits[:before] = float("nan")
    offsets = before + np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    l, t = as_numpy(logits), tokens.cpu().numpy()
    counted = t.copy()
    counted[:before], counted[rows - behind:] = -1, -1
    lp, _ = ref.logprobs(l, counted)
    refs = (torch.from_numpy(lp).to(logits.device) + 0.3 * torch.randn(rows, generator=g, device=logits.device)).float() if with_ref else None
    loss, margins, slopes = ref.preference(lp, counted, offsets, None if refs is None else as_numpy(refs), how.get("beta", 0.1),
                                           how.get("label_smoothing", 0.0), how.get("margin", 0.0), how.get("average", False))
    r = pk.preference_loss(logits, tokens, torch.from_numpy(offsets).to(logits.device), ref_logprobs=refs, **how)
    x, mean = sizes(np.where(np.isnan(l), 0.0, l), 1.0)
    at = np.take_along_axis(x, np.clip(t, 0, n - 1)[:, None], 1)[:, 0]
    live = counted >= 0
    d = np.where(live, row_error(mean, at, lp), 0.0)
    close(as_numpy(r.logprobs), lp, d, "logprobs")
    beta = abs(how.get("beta", 0.1))
    each = np.array([d[a:b].sum() / (max(1, live[a:b].sum()) if how.get("average") else 1) for a, b in zip(offsets[:-1], offsets[1:])])
    dm = beta * (each[0::2] + each[1::2]) + 2.0 ** -23 * np.abs(margins) + 2.0 ** -126
    close(as_numpy(r.margins), margins, dm, "margins")
    pairs = len(lengths) // 2
    close(as_numpy(r.loss), loss, dm.mean() + 2.0 ** -21 * abs(loss) if pairs else 0, "loss")  # a term's slope is at most 1
    # The slope's is at most 1/4; its own operations are a few steps of terms of size beta / pairs.
    ds = np.zeros(rows)
    for j, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
        ds[a:b] = beta / pairs * (dm[j // 2] / 4 + 2.0 ** -21)
    ds = np.where(live, ds, 0.0)
    close(as_numpy(r.slopes), slopes, ds, "slopes")
    gl = torch.full((), scale, device=logits.device)
    grad = ref.gradient(l, counted, 1.0, scale * slopes)
    got = pk.preference_loss_backward(logits, tokens, r, grad_loss=gl)
    off = gradient_error(np.where(np.isnan(l), 0.0, l), 1.0, scale * slopes, None, grad, dtype)
    p = np.exp(-x) / np.exp(-x).sum(1, keepdims=True)
    close(as_numpy(got), grad, off + scale * ds[:, None] * (p + (np.arange(n) == t[:, None])), "gradient")
    assert (got[torch.from_numpy(~live).to(got.device)] == 0).all()
    return logits, tokens, offsets, refs, r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,n,ld", [([1, 1], 7, 0), ([5, 9], 64, 65), ([0, 4, 3, 0], 130, 0), ([0, 0], 50, 0), ([20, 31, 1, 40, 64, 5], 513, 0),
                                          ([3, 5, 2, 2], 5001, 0), ([7, 4], 12000, 12001)])
def test_preference_sizes(pk, cuda_device, dtype, lengths, n, ld):
    check_preference(pk, lengths, n, dtype, ld=ld, scale=16.0)
    check_preference(pk, lengths, n, dtype, ld=ld, before=2, behind=3, scale=16.0)


@pytest.mark.parametrize("how", [dict(beta=1.0), dict(beta=-0.5), dict(beta=0.0), dict(label_smoothing=0.2), dict(label_smoothing=1.0), dict(margin=2.0),
                                 dict(average=True, beta=2.0), dict(average=True, beta=2.5, margin=0.7, label_smoothing=0.1, with_ref=False),
                                 dict(with_ref=False)])
def test_preference_terms(pk, cuda_device, how):
    check_preference(pk, [12, 9, 30, 7, 1, 0], 300, torch.float32, **how)


@pytest.mark.parametrize("pairs", [1, 7, 8, 31, 32, 33, 300])
def test_numbers_of_pairs(pk, cuda_device, pairs):
    rng = np.random.default_rng(pairs)
    check_preference(pk, rng.integers(0, 9, 2 * pairs).tolist(), 40, torch.float32, behind=4)


def test_long_answers(pk, cuda_device):
    check_preference(pk, [3000, 2777], 64, torch.float32)


def test_far_margins(pk, cuda_device):
    # Where one side of the sigmoid is 0 or 1 in float32, and beyond what its exponential holds.
    for beta in (30.0, -30.0, 1000.0, -1000.0):
        check_preference(pk, [30, 20, 9, 9], 50, torch.float32, beta=beta, left_out=0.0, label_smoothing=0.25)
        check_preference(pk, [30, 20, 9, 9], 50, torch.float32, beta=beta, left_out=0.0)


def test_bad_offsets_are_loud_and_harmless(pk, cuda_device):
    logits, tokens, _ = make(20, 100, torch.float32)
    for bad in ([0, 5, 3, 8, 20], [0, 5, 10, 15, 21], [-1, 5, 10, 15, 20], [0, 5, 10, 1 << 40, 20], [-(1 << 62), 1 << 62, 0, 1, 2]):
        r = pk.preference_loss(logits, tokens, torch.tensor(bad, device=cuda_device))
        assert r.loss.isnan() and r.margins.isnan().any()
        pk.preference_loss_backward(logits, tokens, r)
    r = pk.preference_loss(logits, tokens, torch.zeros(1, dtype=torch.int64, device=cuda_device))  # no pair
    assert r.loss == 0 and r.margins.shape == (0,) and (r.slopes == 0).all()
    for bad in (torch.zeros(2, dtype=torch.int64), torch.zeros(0, dtype=torch.int64), torch.zeros((1, 3), dtype=torch.int64)):
        with pytest.raises(ValueError, match="offsets"):
            pk.preference_loss(logits, tokens, bad.to(cuda_device))


def test_preference_autograd(pk, cuda_device):
    logits, tokens, offsets, refs, r = check_preference(pk, [12, 9, 30, 7], 300, torch.float32)
    leaf = logits.clone().requires_grad_()
    o = torch.from_numpy(offsets).to(cuda_device)
    again = pk.preference_loss(leaf, tokens, o, ref_logprobs=refs)
    assert torch.equal(again.loss, r.loss) and again.loss.requires_grad and not again.margins.requires_grad
    (2 * again.loss).backward()
    two = torch.full((), 2.0, device=cuda_device)
    assert torch.equal(leaf.grad, pk.preference_loss_backward(logits, tokens, r, grad_loss=two))
    with pytest.raises(ValueError, match="constant"):
        pk.preference_loss(leaf, tokens, o, ref_logprobs=refs.clone().requires_grad_())


@pytest.mark.parametrize("n", [200, 20000])
def test_streams_and_graphs(pk, cuda_device, n):
    logits, tokens, old, A, refs, w, _, _ = policy_inputs(24, n, torch.bfloat16)
    offsets = torch.tensor([0, 6, 11, 18, 24], device=cuda_device)

    def calls(stream=None):
        a = pk.policy_loss(logits, tokens, old, A, ref_logprobs=refs, weights=w, kl=0.1, entropy=0.1, gradient=True, stream=stream)
        b = pk.preference_loss(logits, tokens, offsets, ref_logprobs=refs, stream=stream)
        return a.loss, a.grad_logits, a.slopes, b.loss, b.margins, pk.preference_loss_backward(logits, tokens, b, stream=stream)
    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = calls(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(calls())
    logits.copy_(logits.flip(0))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for stream, graph in zip(streams, graphs):  # two captured calls side by side
        with torch.cuda.stream(stream):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    want = calls()
    for out in outs:
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_equal_calls_give_equal_bits(pk, cuda_device):
    for rows, n in ((3000, 90), (40, 9000)):
        logits, tokens, old, A, refs, w, _, _ = policy_inputs(rows, n, torch.float16)
        offsets = torch.arange(0, rows + 1, rows // 4, device=cuda_device)[:5]
        first = None
        for _ in range(4):
            r = pk.policy_loss(logits, tokens, old, A, ref_logprobs=refs, weights=w, kl=0.1, entropy=0.1, gradient=True)
            q = pk.preference_loss(logits, tokens, offsets, ref_logprobs=refs)
            now = [*r[:4], r.grad_logits, r.slopes, q.loss, q.margins, q.slopes]
            first = first or now
            assert all(torch.equal(a, b) for a, b in zip(now, first))


def test_messages(pk, cuda_device):
    z, t, _ = make(10, 16, torch.float32)
    one = torch.ones(10, device=cuda_device)
    r = pk.policy_loss(z, t, one, one)
    for call, error, words in (
            (lambda: pk.policy_loss(z, t, one[:3], one), ValueError, r"old_logprobs must have shape \(10,\), not \(3,\)"),
            (lambda: pk.policy_loss(z, t, one, None), TypeError, "advantages"),
            (lambda: pk.policy_loss(z, t, one, one.double()), TypeError, "advantages must be a Float"),
            (lambda: pk.policy_loss(z, t, one, one, out=z), ValueError, "gradient=True"),
            (lambda: pk.policy_loss(z, t, one, one, clip_low=-0.1), pk.ProfkError, ""),
            (lambda: pk.policy_loss(z, t, one, one, kl=float("nan")), pk.ProfkError, ""),
            (lambda: pk.policy_loss(z, t, one, one, gradient=True, out=z.half()), TypeError, "out must be"),
            (lambda: pk.policy_loss_backward(z, t, r, grad_loss=one), ValueError, "one element"),
            (lambda: pk.preference_loss(z, t, torch.zeros(3, dtype=torch.int32, device=cuda_device)), TypeError, "offsets must be a Long"),
            (lambda: pk.preference_loss(z, t, torch.zeros(3, dtype=torch.int64, device=cuda_device), label_smoothing=1.5), pk.ProfkError, ""),
            (lambda: pk.preference_loss(z, t, torch.zeros(3, dtype=torch.int64, device=cuda_device), beta=INF), pk.ProfkError, "")):
        with pytest.raises(error, match=words):
            call()


def test_rows_longer_than_shared_memory(pk, cuda_device):
    # Beyond 8 x 112 KB a row is read twice.
    check_policy(pk, 2, 500_001, torch.bfloat16)
    check_policy(pk, 3, 240_000, torch.float32, with_ref=False, entropy=None)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [3, 700])
def test_rows_kept_whole_and_in_parts(pk, cuda_device, dtype, rows):
    # Sizes about those at which the number of CTAs a row or of their threads changes.
    for n in (8191, 8193, 16384, 16400, 33000, 65536) if rows == 3 else (4097, 8190, 8200, 16390):
        check_policy(pk, rows, n, dtype, left_out=0.1, entropy=None)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_logits_and_sharp_temperatures(pk, cuda_device, dtype):
    for n in (300, 9001, 40000):
        check_policy(pk, 7, n, dtype, T=0.02, kl=0.0, with_ref=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [300, 9001])
@pytest.mark.parametrize("T", [1e-3, 1.0, 900.0, 1e5])
def test_masked_logits_at_all_temperatures(pk, cuda_device, dtype, n, T):
    # -inf, and the type's lowest value, at temperatures at which a bounded stand-in would or would not have mass.
    logits, tokens, g = make(8, n, dtype, spread=3.0 * min(1.0, T * 10))
    logits[:, n // 3: n // 2] = -INF
    logits[3, n // 2: n // 2 + 9] = torch.finfo(dtype).min
    logits[4, : n // 3] = logits[4, n // 2:] = torch.finfo(dtype).min
    tokens.fill_(n - 1)
    h = torch.full((8,), 1000.0, device=cuda_device)
    dg = torch.randn(8, generator=g, device=cuda_device)
    r = pk.token_logprobs(logits, tokens, temperature=T, entropy=True)
    got = pk.token_logprobs_backward(logits, tokens, r, grad_logprobs=dg, grad_entropies=h)
    assert not got.isnan().any() and not r.entropies.isnan().any()
    l, t = as_numpy(logits), tokens.cpu().numpy()
    lp, H = ref.logprobs(l, t, T)
    x, mean = sizes(l, T)
    at = np.take_along_axis(x, t[:, None], 1)[:, 0]
    close(as_numpy(r.logprobs), lp, row_error(mean, at, lp))
    close(as_numpy(r.entropies), H, row_error(mean, value=H) + 2.0 ** -18 * mean)
    want = ref.gradient(l, t, T, as_numpy(dg), as_numpy(h))
    # An entropy's slope takes the mean of x as log s - H, each with its rounding: 2^-22 of their sizes.
    extra = 1000.0 / T * np.where(np.isfinite(l), np.exp(-x), 0.0) / np.exp(-x).sum(1, keepdims=True) * (2.0 ** -21 * (np.log(n) + np.abs(H)))[:, None]
    off = gradient_error(l, T, as_numpy(dg), as_numpy(h), want, dtype) + extra
    if dtype == torch.float16:  # from 65520 on its rounding is infinite
        want = np.where(np.abs(want) - off > 65520, np.copysign(INF, want), want)
    close(as_numpy(got), want, off)
    assert (got[:, n // 3: n // 2] == 0).all()


def test_margins_of_long_answers(pk, cuda_device):
    # A float32 log-probability is off by up to 2^-23 of 4 to 8 from its rounding alone; the sums take what it lacks along,
    # so that a margin over 2 x 2000 tokens is off by their rows' sums (2^-24 each, of either sign) and not by that.
    logits, tokens, g = make(4000, 700, torch.float16)
    offsets = torch.tensor([0, 2000, 4000], device=cuda_device)
    lp, _ = ref.logprobs(as_numpy(logits), tokens.cpu().numpy())
    r = pk.preference_loss(logits, tokens, offsets, beta=1.0)
    want = lp[:2000].sum() - lp[2000:].sum()
    assert abs(r.margins.item() - want) < 2.0 ** -24 * abs(want) + 4000 ** 0.5 * 2.0 ** -23
