"""route and route_backward against their definitions in float64 (oracle/selections.py).

The choice is a comparison of float32 numbers, so experts and counts are equal.
Gates: an exponential's argument carries two roundings of a number below 2^5
(2^-18.4 relative with room), the exponential, the sum and the quotient an ulp
or two each: 1e-5 relative.  The loss is a mean of such numbers.  Gradients are
sums of at most four such terms, each bounded by the token's largest |dg| and
the balance term, plus one rounding to the logits' type.
"""
import numpy as np
import pytest
import torch

from oracle import selections as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -24}


def inputs(tokens, E, dtype, seed, device, ld=None, offset=0, spread=1.5):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    ld = ld or E
    store = torch.empty(tokens * ld + offset, dtype=dtype, device=device).fill_(torch.finfo(dtype).max)
    z = store[offset:].view(tokens, ld)[:, :E]
    z.copy_(spread * torch.randn((tokens, E), generator=g, device=device))
    return z, g


def check(pk, z, k, score, normalize, bias=None, mask=None, backward=True, seed=0):
    r = pk.route(z, k, score=score, normalize=normalize, bias=bias, mask=mask)
    bare = pk.route(z, k, score=score, normalize=normalize, bias=bias, mask=mask, balance=False)
    assert bare.loss is None and all(torch.equal(a, b) for a, b in ((bare.experts, r.experts), (bare.counts, r.counts)))
    assert torch.equal(bare.gates.view(torch.int32), r.gates.view(torch.int32))
    z32 = z.float().cpu().numpy()
    np_of = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    gates, experts, counts, loss = ref.routing(z32, k, score, normalize, np_of(bias), np_of(mask))
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    np.testing.assert_allclose(r.gates.cpu().numpy(), gates, rtol=1e-5, atol=1e-12)
    np.testing.assert_allclose(r.loss.item(), loss, rtol=1e-5, atol=1e-12)
    if backward:
        g = torch.Generator(device=z.device)
        g.manual_seed(seed + 1)
        dg = torch.randn(r.gates.shape, generator=g, device=z.device)
        dl = torch.tensor(0.7 * z.shape[0], device=z.device)
        for use_g, use_l in ((True, True), (True, False), (False, True)):
            got = pk.route_backward(z, r, grad_gates=dg if use_g else None, grad_loss=dl if use_l else None)
            again = pk.route_backward(z, r, grad_gates=dg if use_g else None, grad_loss=dl if use_l else None)
            assert got.dtype == z.dtype and torch.equal(got, again)
            want = ref.routing_gradient(z32, experts, counts, score, normalize, np_of(dg) if use_g else None,
                                        dl.item() if use_l else None)
            E, N = z.shape[1], max(counts.sum(), 1)
            size = np.zeros((z.shape[0], 1))
            if use_g:
                size += np.abs(np_of(dg)).max(1, keepdims=True)
            if use_l:
                size += dl.item() * E * counts.max() / N * k / N
            tol = 1e-5 * size + EPS[z.dtype] * np.abs(want) + TINY[z.dtype]
            off = np.abs(got.double().cpu().numpy() - want) - tol
            assert (off <= 0).all(), (off.max(), use_g, use_l)
    return r


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,E,k", [(1, 8, 2), (7, 60, 4), (300, 128, 8), (1000, 256, 8), (33, 511, 7)])
def test_forms(pk, cuda_device, tokens, E, k, dtype, score, normalize):
    z, g = inputs(tokens, E, dtype, tokens, cuda_device)
    check(pk, z, k, score, normalize)
    bias = torch.randn(E, generator=g, device=cuda_device)
    mask = torch.rand(tokens, generator=g, device=cuda_device) < 0.7
    check(pk, z, k, score, normalize, bias=bias, mask=mask)


@pytest.mark.parametrize("E", [1, 2, 3, 5, 8, 16, 31, 32, 33, 63, 64, 65, 96, 127, 129, 160, 255, 257, 384, 512, 513, 1023, 1024])
def test_expert_counts(pk, cuda_device, E):
    for dtype in TYPES:
        z, _ = inputs(50, E, dtype, E, cuda_device)
        for k in sorted({1, min(E, 2), min(E, 6), min(E, 32)}):
            check(pk, z, k, "softmax" if k % 2 else "sigmoid", True)


@pytest.mark.parametrize("k", list(range(1, 33)))
def test_slots(pk, cuda_device, k):
    z, _ = inputs(40, 40, torch.bfloat16, k, cuda_device)
    check(pk, z, k, "softmax", k % 2 == 0)


@pytest.mark.parametrize("tokens", [0, 1, 2, 8, 9, 151, 152, 153, 1217, 5000, 40000])
def test_token_counts(pk, cuda_device, tokens):
    z, _ = inputs(tokens, 24, torch.bfloat16, 3, cuda_device)
    if tokens == 0:
        r = pk.route(z, 2)
        assert r.loss.item() == 0 and (r.counts == 0).all() and r.gates.shape == (0, 2)
        assert pk.route_backward(z, r, grad_loss=torch.ones((), device=cuda_device)).shape == (0, 24)
        return
    check(pk, z, 3, "softmax", True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,ld,offset", [(64, 64, 1), (64, 65, 0), (64, 72, 8), (60, 61, 3), (128, 136, 4)])
def test_strides_and_alignment(pk, cuda_device, dtype, E, ld, offset):
    z, _ = inputs(100, E, dtype, 5, cuda_device, ld=ld, offset=offset)
    r = check(pk, z, 4, "softmax", True)
    wide = torch.full((100, E + 9), 7.0, dtype=dtype, device=cuda_device)
    dg = torch.ones_like(r.gates).cumsum(1)
    got = pk.route_backward(z, r, grad_gates=dg, out=wide[:, 3:3 + E])
    assert torch.equal(got, pk.route_backward(z, r, grad_gates=dg)) and (wide[:, :3] == 7).all() and (wide[:, 3 + E:] == 7).all()


def test_rows_far_apart(pk, cuda_device):
    # Offsets of logits and their gradient past 2^31 elements.
    E, far = 100, (1 << 30) + 512
    z = torch.randn((4, E), device=cuda_device).to(torch.bfloat16)
    store, grad = (torch.empty(3 * far + E, dtype=torch.bfloat16, device=cuda_device).as_strided((4, E), (far, 1))
                   for _ in range(2))
    store.copy_(z)
    want, got = pk.route(z, 5), pk.route(store, 5)
    assert all(torch.equal(getattr(got, f), getattr(want, f)) for f in ("gates", "experts", "counts", "loss"))
    dg, dl = torch.randn_like(got.gates), torch.ones((), device=cuda_device)
    pk.route_backward(store, got, grad_gates=dg, grad_loss=dl, out=grad)
    assert torch.equal(grad, pk.route_backward(z, want, grad_gates=dg, grad_loss=dl))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
def test_special_values(pk, cuda_device, dtype, score, normalize):
    z, _ = inputs(12, 48, dtype, 8, cuda_device)
    inf, low = float("inf"), torch.finfo(dtype).min
    z[0] = -inf            # nothing to choose: as a masked token
    z[1, 3:] = -inf        # fewer than k
    z[2] = 0.0             # ties: the lowest indices
    z[3, ::2] = -0.0
    z[3, 1::2] = 0.0
    z[4] = low             # the lowest value of the type is a value
    z[5, 5:] = low
    z[6] = 80.0            # sigmoid: all 1 - 2^-115
    z[7] = -80.0           # sigmoid: all underflowing in a plain product
    z[8, 7] = 60.0
    r = check(pk, z, 6, score, normalize)
    e = r.experts.cpu()
    assert (e[0] == -1).all() and (e[1, 3:] == -1).all() and e[1, :3].min() >= 0
    assert e[2].tolist() == e[3].tolist() == e[4].tolist() == list(range(6))


def test_infinite_and_nan_logits(pk, cuda_device):
    z, _ = inputs(6, 40, torch.float32, 9, cuda_device)
    inf, nan = float("inf"), float("nan")
    z[1, [4, 9]] = inf
    z[2, 17] = nan
    z[3] = nan
    mask = torch.tensor([True, True, True, False, True, True], device=cuda_device)
    for normalize in (True, False):
        check(pk, z, 4, "softmax", normalize, mask=torch.tensor([1, 1, 0, 0, 1, 1], dtype=torch.bool, device=cuda_device),
              backward=False)
        r = pk.route(z, 4, normalize=normalize, mask=mask)
        assert r.experts[1, :2].tolist() == [4, 9] and r.gates[1].tolist() == [0.5, 0.5, 0, 0]
        assert torch.isnan(r.gates[2]).all() and 17 not in r.experts[2].tolist() and (r.experts[2] >= 0).all()
        assert (r.experts[3] == -1).all() and (r.gates[3] == 0).all() and torch.isnan(r.loss)
        d = pk.route_backward(z, r, grad_gates=torch.ones_like(r.gates))
        assert (d[3] == 0).all() and torch.isfinite(d[[0, 1, 4, 5]]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_a_negative_nan_is_a_nan(pk, cuda_device, dtype):
    z, _ = inputs(4, 40, dtype, 19, cuda_device)
    bits = {torch.float32: (torch.int32, -0x400000), torch.bfloat16: (torch.int16, -0x40), torch.float16: (torch.int16, -0x200)}
    kind, value = bits[dtype]
    z.view(kind)[2, 11] = value
    assert torch.isnan(z[2, 11])
    for bias in (None, torch.zeros(40, device=cuda_device)):
        r = pk.route(z, 5, bias=bias)
        assert torch.isnan(r.gates[2]).all() and torch.isnan(r.loss) and 11 not in r.experts[2].tolist()
        assert (r.experts >= 0).all() and torch.isfinite(r.gates[[0, 1, 3]]).all()


def test_a_bias_chooses_only(pk, cuda_device):
    z, _ = inputs(64, 32, torch.float32, 10, cuda_device)
    bias = torch.zeros(32, device=cuda_device)
    bias[7] = 1000.0
    bias[3] = float("-inf")
    for score in ("softmax", "sigmoid"):
        z[0, 7] = -200.0  # its gate stays that of a score of exp(-200)
        r = check(pk, z, 3, score, True, bias=bias)
        assert (r.experts[:, 0] == 7).all() and (r.experts != 3).all()
        z[1] = -150.0
        check(pk, z, 3, score, True, bias=bias)


def test_every_token_masked(pk, cuda_device):
    z, _ = inputs(9, 16, torch.bfloat16, 11, cuda_device)
    r = pk.route(z, 2, mask=torch.zeros(9, dtype=torch.bool, device=cuda_device))
    assert (r.experts == -1).all() and (r.gates == 0).all() and (r.counts == 0).all() and r.loss.item() == 0
    d = pk.route_backward(z, r, grad_gates=torch.ones_like(r.gates), grad_loss=torch.ones((), device=cuda_device))
    assert (d == 0).all()


def test_balance(pk, cuda_device):
    # Every expert the same share: 1.  All to one expert that also has the mass: E.
    E = 16
    z = torch.full((E * 8, E), -30.0, device=cuda_device)
    z[torch.arange(E * 8), torch.arange(E * 8) % E] = 30.0
    r = pk.route(z, 1)
    assert abs(r.loss.item() - 1) < 1e-6 and (r.counts == 8).all()
    z[:] = -30.0
    z[:, 5] = 30.0
    assert abs(pk.route(z, 1).loss.item() - E) < 1e-5


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(pk, cuda_device, score, normalize):
    # Along random unit directions per token, h = 2^-6: the third derivative of these functions is
    # below the sum of |dg| and the loss's slope (h^2 / 6 of it), rounding is 2^-23 of them / h.
    tokens, E, k = 16, 24, 4
    z, g = inputs(tokens, E, torch.float32, 12, cuda_device)
    z += 0.3 * torch.arange(E, device=cuda_device) % 7  # no two of a token's logits swap within h
    r = pk.route(z, k, score=score, normalize=normalize)
    dg = torch.randn(r.gates.shape, generator=g, device=cuda_device)
    dl = torch.tensor(2.0 * tokens, device=cuda_device)
    grad = pk.route_backward(z, r, grad_gates=dg, grad_loss=dl).double()
    h, done = 2.0 ** -6, 0
    for _ in range(12):
        v = torch.randn(z.shape, generator=g, device=cuda_device)
        v /= v.norm(dim=1, keepdim=True)
        a, b = (pk.route(z + s * h * v, k, score=score, normalize=normalize) for s in (1, -1))
        if not (torch.equal(a.experts, r.experts) and torch.equal(b.experts, r.experts)):
            continue  # the choice is not a constant along this direction
        done += 1
        f = [((x.gates.double() * dg).sum() + x.loss.double() * dl).item() for x in (a, b)]
        slope = (f[0] - f[1]) / (2 * h)
        size = dg.abs().sum().item() + dl.item()
        assert abs(slope - (grad * v).sum().item()) < size * (h * h / 6 + 2.0 ** -23 / h), (score, normalize)
    assert done >= 1


def test_autograd(pk, cuda_device):
    z, g = inputs(200, 64, torch.bfloat16, 13, cuda_device)
    w = torch.randn((200, 6), generator=g, device=cuda_device)
    leaf = z.clone().requires_grad_()
    r = pk.route(leaf, 6)
    ((r.gates * w).sum() + 3 * r.loss).backward()
    plain = pk.route(z, 6)
    want = pk.route_backward(z, plain, grad_gates=w, grad_loss=torch.tensor(3.0, device=cuda_device))
    assert torch.equal(leaf.grad, want)
    leaf.grad = None
    r = pk.route(leaf, 6, balance=False)
    assert r.loss is None
    (r.gates * w).sum().backward()
    assert torch.equal(leaf.grad, pk.route_backward(z, plain, grad_gates=w))
    leaf.grad = None
    pk.route(leaf, 6).loss.backward()
    assert torch.equal(leaf.grad, pk.route_backward(z, plain, grad_loss=torch.ones((), device=cuda_device)))
    with pytest.raises(ValueError):
        pk.route(leaf, 6, stream=torch.cuda.Stream())
    with torch.no_grad():
        assert not pk.route(leaf, 6).gates.requires_grad


def test_counts_summed_over_devices(pk, cuda_device):
    # Two halves with the sum of their counts: the halves of the whole batch's gradient.
    z, _ = inputs(128, 32, torch.float32, 14, cuda_device)
    whole = pk.route(z, 4)
    dl = torch.tensor(50.0, device=cuda_device)
    want = pk.route_backward(z, whole, grad_loss=dl)
    for half in (slice(0, 64), slice(64, 128)):
        r = pk.route(z[half], 4)._replace(counts=whole.counts)
        got = pk.route_backward(z[half], r, grad_loss=dl)
        assert torch.equal(got, want[half])


def test_foreign_choices(pk, cuda_device):
    # Entries outside [0, experts) are empty slots, whatever they hold.
    z, _ = inputs(20, 16, torch.float32, 15, cuda_device)
    r = pk.route(z, 3)
    odd = r.experts.clone()
    odd[3, 1], odd[4, 0], odd[5] = 16, -(1 << 40), 1 << 50
    dg = torch.ones_like(r.gates).cumsum(1)
    got = pk.route_backward(z, r._replace(experts=odd), grad_gates=dg).double().cpu().numpy()
    want = ref.routing_gradient(z.cpu().numpy(), odd.cpu().numpy(), r.counts.cpu().numpy(), "softmax", True,
                                dg.cpu().numpy())
    assert np.abs(got - want).max() < 3e-5 and (got[5] == 0).all()


def test_streams_and_graph(pk, cuda_device):
    z, _ = inputs(2000, 64, torch.bfloat16, 16, cuda_device)
    want = pk.route(z, 4)
    dg = torch.ones_like(want.gates).cumsum(1)
    dz = pk.route_backward(z, want, grad_gates=dg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = pk.route(z, 4, stream=side)
    d = pk.route_backward(z, r, grad_gates=dg, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(r[:4], want[:4])) and torch.equal(d, dz)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = pk.route(z, 4)
        d = pk.route_backward(z, r, grad_gates=dg)
    z.copy_(z.flip(0))
    graph.replay()
    want = pk.route(z, 4)
    assert all(torch.equal(a, b) for a, b in zip(r[:4], want[:4]))
    assert torch.equal(d, pk.route_backward(z, want, grad_gates=dg))


def test_refusals(pk, cuda_device):
    z, _ = inputs(10, 16, torch.float32, 17, cuda_device)
    with pytest.raises(TypeError):
        pk.route(z.double(), 2)
    with pytest.raises(TypeError):
        pk.route(z.cpu(), 2)
    with pytest.raises(ValueError):
        pk.route(z[0], 2)
    with pytest.raises(ValueError):
        pk.route(z.t(), 2)
    for k in (0, 17):
        with pytest.raises(ValueError):
            pk.route(z, k)
    with pytest.raises(ValueError):
        pk.route(z, 2, score="tanh")
    with pytest.raises(ValueError):
        pk.route(z, 2, bias=torch.zeros(15, device=cuda_device))
    with pytest.raises(TypeError):
        pk.route(z, 2, bias=torch.zeros(16, device=cuda_device, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        pk.route(z, 2, mask=torch.ones(10, device=cuda_device))
    for E, k in ((1025, 2), (64, 33)):
        with pytest.raises(pk.ProfkError) as e:
            pk.route(torch.zeros((2, E), device=cuda_device), k)
        assert e.value.code == -4
    r = pk.route(z, 2)
    with pytest.raises(ValueError):
        pk.route_backward(z, r, grad_gates=torch.zeros((10, 3), device=cuda_device))
    with pytest.raises(TypeError):
        pk.route_backward(z, r, grad_gates=torch.zeros((10, 2), device=cuda_device, dtype=torch.float64))
    with pytest.raises(ValueError):
        pk.route_backward(z, r, grad_loss=torch.zeros(2, device=cuda_device))
    with pytest.raises(TypeError):
        pk.route_backward(z, r, out=torch.zeros((10, 16), device=cuda_device, dtype=torch.float16))
    with pytest.raises(ValueError):
        pk.route_backward(z[:5], r)
