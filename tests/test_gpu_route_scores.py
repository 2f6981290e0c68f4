"""route with the bias added to the scores, against the definition in float64 (oracle/selections.py).

The choice is a comparison of float32 numbers score + bias.  A score's exponential
has an argument of two roundings and two ulps of its own, its sum and quotient an
ulp or two: below 2^-21 of a number of at most 1, and the sum's rounding is 2^-24
of itself.  Experts whose exact numbers differ by less than 2^-20 (1 + |c|) may
come in either order; those with the same logit and bias come by index.  What
follows from the choice has the tolerances of test_gpu_route.py.
"""
import numpy as np
import pytest
import torch

from oracle import selections as ref
from test_gpu_route import EPS, TINY, TYPES, inputs

pytestmark = pytest.mark.gpu


def check(pk, z, k, score, normalize, bias, mask=None, backward=True, most_unclear=0.05):
    r = pk.route(z, k, score=score, normalize=normalize, bias=bias, mask=mask, bias_on="scores")
    again = pk.route(z, k, score=score, normalize=normalize, bias=bias, mask=mask, bias_on="scores", balance=False)
    assert torch.equal(r.experts, again.experts) and torch.equal(r.gates, again.gates) and again.loss is None
    z32, b, e = z.float().cpu().numpy(), bias.cpu().numpy(), r.experts.cpu().numpy()
    c = ref.scores_and_bias(z32, score, b)
    c = np.where(np.isnan(c), -np.inf, c)
    unclear = 0
    for t in range(len(z32)):
        order = ref.order_of(c[t]) if mask is None or mask[t] else ref.order_of(c[t])[:0]
        filled = min(k, order.size)
        got = e[t, :filled]
        assert (e[t, filled:] == -1).all() and len(set(got.tolist())) == filled and np.isin(got, order).all()
        if np.array_equal(got, order[:filled]):
            continue
        unclear += 1
        blur = 2.0 ** -20 * (1 + np.abs(c[t][order]).max())
        rest = np.setdiff1d(order, got)
        run = np.concatenate([c[t][got], [c[t][rest].max() if rest.size else -np.inf]])
        assert (run[1:] - run[:-1] <= blur).all(), (t, got, order[:filled])
        after = np.concatenate([got, np.sort(rest)])
        for i, j in zip(after[:-1], after[1:]):  # neighbours with one logit and bias
            if z32[t, i] == z32[t, j] and b[i] == b[j]:
                assert i < j
    assert unclear <= max(1, most_unclear * len(z32)), unclear
    gates, counts, loss = ref.routed(z32, e, score, normalize)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    np.testing.assert_allclose(r.gates.cpu().numpy(), gates, rtol=1e-5, atol=1e-12)
    np.testing.assert_allclose(r.loss.item(), loss, rtol=1e-5, atol=1e-12)
    if backward:
        g = torch.Generator(device=z.device)
        g.manual_seed(7)
        dg = torch.randn(r.gates.shape, generator=g, device=z.device)
        dl = torch.tensor(0.7 * len(z32), device=z.device)
        got = pk.route_backward(z, r, grad_gates=dg, grad_loss=dl).double().cpu().numpy()
        dg = dg.cpu().numpy()
        want = ref.routing_gradient(z32, e, counts, score, normalize, dg, dl.item())
        N = max(counts.sum(), 1)
        size = np.abs(dg).max(1, keepdims=True) + dl.item() * z32.shape[1] * counts.max() / N * k / N
        assert (np.abs(got - want) <= 1e-5 * size + EPS[z.dtype] * np.abs(want) + TINY[z.dtype]).all()
    return r


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,E,k", [(1, 8, 2), (7, 60, 4), (300, 128, 8), (1000, 256, 8), (33, 511, 7), (600, 40, 32)])
def test_forms(pk, cuda_device, tokens, E, k, dtype, score, normalize):
    z, g = inputs(tokens, E, dtype, tokens, cuda_device)
    bias = 0.3 * torch.randn(E, generator=g, device=cuda_device)
    check(pk, z, k, score, normalize, bias)
    check(pk, z, k, score, normalize, bias, mask=torch.rand(tokens, generator=g, device=cuda_device) < 0.7)


@pytest.mark.parametrize("E", [1, 2, 31, 33, 64, 65, 128, 129, 257, 513, 1024])
def test_expert_counts(pk, cuda_device, E):
    for dtype in TYPES:
        z, g = inputs(700 if E > 500 else 50, E, dtype, E, cuda_device)
        bias = 0.1 * torch.randn(E, generator=g, device=cuda_device)
        for k in sorted({1, min(E, 6), min(E, 32)}):
            check(pk, z, k, "softmax" if k % 2 else "sigmoid", True, bias, backward=False)


def test_the_two_rules_differ(pk, cuda_device):
    z = torch.tensor([[2.0, 0.0]], device=cuda_device)
    bias = torch.tensor([0.0, 0.6], device=cuda_device)
    assert pk.route(z, 1, score="sigmoid", bias=bias).experts.item() == 0                       # 2 against 0.6
    r = pk.route(z, 1, score="sigmoid", normalize=False, bias=bias, bias_on="scores")           # 0.88 against 1.10
    assert r.experts.item() == 1 and abs(r.gates.item() - 0.5) < 1e-6
    bias = torch.tensor([0.0, 0.9], device=cuda_device)
    r = pk.route(z, 1, normalize=False, bias=bias, bias_on="scores")                            # 0.88 against 0.12 + 0.9
    assert r.experts.item() == 1 and abs(r.gates.item() - 1 / (1 + np.e ** 2)) < 1e-6
    assert pk.route(z, 1, bias=bias).experts.item() == 0


def test_without_a_bias_it_does_not_matter(pk, cuda_device):
    z, _ = inputs(700, 96, torch.bfloat16, 3, cuda_device)
    for score in ("softmax", "sigmoid"):
        a, b = (pk.route(z, 5, score=score, bias_on=on) for on in ("logits", "scores"))
        assert all(torch.equal(x, y) for x, y in zip(a[:4], b[:4]))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
def test_special_values(pk, cuda_device, dtype, score):
    z, g = inputs(12, 48, dtype, 8, cuda_device)
    inf, low = float("inf"), torch.finfo(dtype).min
    z[0] = -inf            # nothing to choose
    z[1, 3:] = -inf        # fewer than k, whatever their bias
    z[2] = 0.0             # ties
    z[3, ::2], z[3, 1::2] = -0.0, 0.0
    z[4] = low             # the lowest value of the type is a value
    z[5, 5:] = low
    z[6] = 80.0            # scores of 1
    z[7] = -200.0          # sigmoid: scores of 0
    z[8, [7, 9]] = 60.0
    bias = torch.zeros(48, device=cuda_device)
    r = check(pk, z, 6, score, True, bias)
    e = r.experts.cpu()
    assert (e[0] == -1).all() and sorted(e[1, :3].tolist()) == [0, 1, 2] and (e[1, 3:] == -1).all()
    assert e[2].tolist() == e[3].tolist() == e[4].tolist() == e[6].tolist() == e[7].tolist() == list(range(6))
    bias[10], bias[11], bias[40] = 5.0, -inf, 1e30
    r = check(pk, z, 6, score, False, bias)
    e = r.experts.cpu()
    assert sorted(e[1, :3].tolist()) == [0, 1, 2] and (e[1, 3:] == -1).all() and not (e == 11).any()
    assert (e[2:, 0] == 40).all() and (e[2:, 1] == 10).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_and_infinite_logits(pk, cuda_device, score):
    z, g = inputs(6, 40, torch.float32, 9, cuda_device)
    inf, nan = float("inf"), float("nan")
    bias = 0.05 * torch.randn(40, generator=g, device=cuda_device)
    z[1, [4, 9]] = inf
    z[2, 17] = nan
    z[3] = nan
    r = pk.route(z, 4, score=score, bias=bias, bias_on="scores")
    without = z.clone()
    without[2, 17] = -inf
    left = pk.route(without[2:3], 4, score=score, bias=bias, bias_on="scores")
    assert torch.equal(r.experts[2:3], left.experts) and torch.isnan(r.gates[2]).all()
    assert (r.experts[3] == -1).all() and (r.gates[3] == 0).all() and torch.isnan(r.loss)
    assert sorted(r.experts[1, :2].tolist()) == [4, 9] and torch.isfinite(r.gates[[0, 1, 4, 5]]).all()


def test_strides_streams_autograd_and_refusals(pk, cuda_device):
    for ld, offset in ((65, 0), (72, 3)):
        z, g = inputs(700, 64, torch.bfloat16, 5, cuda_device, ld=ld, offset=offset)
        bias = 0.2 * torch.randn(64, generator=g, device=cuda_device)
        r = check(pk, z, 4, "sigmoid", True, bias)
    w = torch.randn(r.gates.shape, generator=g, device=cuda_device)
    leaf = z.clone().requires_grad_()
    a = pk.route(leaf, 4, score="sigmoid", bias=bias, bias_on="scores")
    assert torch.equal(a.experts, r.experts)
    ((a.gates * w).sum() + 3 * a.loss).backward()
    assert torch.equal(leaf.grad, pk.route_backward(z, r, grad_gates=w, grad_loss=torch.tensor(3.0, device=cuda_device)))
    with pytest.raises(ValueError, match="bias_on"):
        pk.route(z, 4, bias=bias, bias_on="gates")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = pk.route(z, 4, score="sigmoid", bias=bias, bias_on="scores", stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(b[:4], r[:4]))
