"""The log-probability calls without a GPU: argument checks of the C-ABI (made before any device work), the float64
definitions that the GPU tests use, and the place in autograd."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import logprobs as ref

P, ODD, FOUR = C.c_void_p(256), C.c_void_p(257), C.c_void_p(260)
NAN, INF = float("nan"), float("inf")


@pytest.fixture()
def lib(pk):
    return pk.lib()


def status():
    from streaming_selection_primitive_gb300 import _abi
    return _abi.PROFK_ERR_INVALID, _abi.PROFK_ERR_UNSUPPORTED


ROWS_INVALID = [{"kind": 3}, {"kind": -1}, {"rows": -1}, {"n": 0}, {"ld": 9}, {"logits": None}, {"tokens": None}] + [
    {"T": t} for t in (0.0, -1.0, NAN, INF, 1e-45, 3e38 * 10)]
ROWS_UNSUPPORTED = [{"n": 1 << 30, "ld": 1 << 30, "grad_ld": 1 << 30}, {"rows": 1 << 28}, {"logits": ODD}, {"tokens": FOUR}, {"temperature": ODD}]


def test_token_logprobs_checks_arguments(lib):
    invalid, unsupported = status()

    def call(logits=P, kind=1, rows=2, n=10, ld=10, tokens=P, temperature=None, T=1.0, lp=P, H=None, stats=P, grad_ld=0):
        return lib.profk_token_logprobs(logits, kind, rows, n, ld, tokens, temperature, T, lp, H, stats, None)

    assert call(rows=0, logits=None, tokens=None, lp=None) == 0
    for bad in ROWS_INVALID + [{"lp": None}]:
        assert call(**bad) == invalid, bad
    for bad in ROWS_UNSUPPORTED + [{"lp": ODD}, {"H": ODD}, {"stats": FOUR}]:
        assert call(**bad) == unsupported, bad


def test_token_logprobs_backward_checks_arguments(lib):
    invalid, unsupported = status()
    far = C.c_void_p(1 << 40)

    def call(logits=P, kind=1, rows=2, n=10, ld=10, tokens=P, temperature=None, T=1.0, stats=P, H=None, g=P, h=None, scale=None,
             grad=far, grad_ld=10):
        return lib.profk_token_logprobs_backward(logits, kind, rows, n, ld, tokens, temperature, T, stats, H, g, h, scale, grad, grad_ld, None)

    assert call(rows=0) == 0
    # Across the logits: one element on, another row stride; before them, their last element.
    across = [{"grad": C.c_void_p(258)}, {"grad": P, "grad_ld": 11}, {"grad": C.c_void_p(256 + 38)}, {"grad": C.c_void_p(256 - 38)}]
    for bad in ROWS_INVALID + [{"stats": None}, {"grad": None}, {"grad_ld": 9}, {"h": P}] + across:
        assert call(**bad) == invalid, bad
    for bad in ROWS_UNSUPPORTED + [{"stats": FOUR}, {"g": ODD}, {"H": ODD, "h": P}, {"H": P, "h": ODD}, {"scale": ODD}, {"grad": C.c_void_p((1 << 40) + 1)}]:
        assert call(**bad) == unsupported, bad


def test_head_logprobs_checks_arguments(lib):
    invalid, unsupported = status()

    def call(hidden=P, weight=P, kind=1, rows=2, n=10, width=16, hld=16, wld=16, tokens=P, temperature=None, T=1.0, lp=P, H=None):
        return lib.profk_head_logprobs(hidden, weight, kind, rows, n, width, hld, wld, tokens, temperature, T, lp, H, None)

    assert call(rows=0) == 0
    for bad in ({"kind": 0}, {"kind": 3}, {"rows": -1}, {"n": 0}, {"width": 0}, {"hld": 8}, {"wld": 15}, {"T": 0.0}, {"T": NAN}, {"hidden": None},
                {"weight": None}, {"tokens": None}, {"lp": None}):
        assert call(**bad) == invalid, bad
    for bad in ({"n": 1 << 30}, {"rows": 1 << 24}, {"width": 1 << 20, "hld": 1 << 20, "wld": 1 << 20}, {"hld": 17}, {"wld": 20}, {"hidden": C.c_void_p(264)},
                {"weight": C.c_void_p(258)}, {"tokens": FOUR}, {"lp": ODD}, {"H": ODD}, {"temperature": ODD}, {"hld": 1 << 38}):
        assert call(**bad) == unsupported, bad


def test_policy_loss_checks_arguments(lib):
    from streaming_selection_primitive_gb300 import _abi
    invalid, unsupported = status()
    fields = dict(old_logprobs=256, advantages=256, clip_low=0.2, clip_high=0.2)

    def call(logits=P, kind=1, rows=2, n=10, ld=10, tokens=P, temperature=None, T=1.0, loss=P, sums=P, lp=P, H=P, stats=P, slopes=P, hs=None,
             grad=None, grad_ld=10, **how):
        return lib.profk_policy_loss(logits, kind, rows, n, ld, tokens, temperature, T, _abi.Policy(**{**fields, **how}), loss, sums, lp, H,
                                     stats, slopes, hs, grad, grad_ld, None)

    for bad in ROWS_INVALID + [{"loss": None}, {"sums": None}, {"lp": None}, {"stats": None}, {"slopes": None}, {"clip_low": -0.1}, {"clip_high": NAN},
                               {"kl": INF}, {"entropy": NAN}, {"entropy": 0.1, "H": None}, {"old_logprobs": None}, {"advantages": None},
                               {"grad": P, "grad_ld": 9}, {"grad": C.c_void_p(258)}]:
        assert call(**bad) == invalid, bad
    for bad in ROWS_UNSUPPORTED + [{"old_logprobs": 257}, {"advantages": 257}, {"ref_logprobs": 257}, {"weights": 258}, {"loss": ODD}, {"sums": ODD},
                                   {"stats": FOUR}, {"slopes": ODD}, {"hs": ODD}, {"grad": C.c_void_p((1 << 40) + 1)}]:
        assert call(**bad) == unsupported, bad


def test_preference_loss_checks_arguments(lib):
    from streaming_selection_primitive_gb300 import _abi
    invalid, unsupported = status()

    def call(logits=P, kind=1, rows=2, n=10, ld=10, tokens=P, temperature=None, T=1.0, offsets=P, pairs=1, loss=P, margins=P, lp=P, stats=P, slopes=P,
             grad_ld=0, **how):
        return lib.profk_preference_loss(logits, kind, rows, n, ld, tokens, temperature, T, offsets, pairs, _abi.Preference(**{"beta": 0.1, **how}),
                                         loss, margins, lp, stats, slopes, None)

    for bad in ROWS_INVALID + [{"offsets": None}, {"pairs": -1}, {"loss": None}, {"margins": None}, {"lp": None}, {"stats": None}, {"slopes": None},
                               {"beta": NAN}, {"margin": INF}, {"label_smoothing": -0.1}, {"label_smoothing": 1.1}, {"label_smoothing": NAN}]:
        assert call(**bad) == invalid, bad
    for bad in ROWS_UNSUPPORTED + [{"offsets": FOUR}, {"pairs": 1 << 28}, {"ref_logprobs": 257}, {"loss": ODD}, {"margins": ODD}, {"slopes": ODD}, {"stats": FOUR}]:
        assert call(**bad) == unsupported, bad


# ---- the definitions ---------------------------------------------------------------------------

def differences(f, l, h=2.0 ** -12):
    out = np.zeros_like(l)
    for i in np.ndindex(l.shape):
        a, b = l.copy(), l.copy()
        a[i] += h
        b[i] -= h
        out[i] = (f(a) - f(b)) / (2 * h)
    return out


def test_gradient_definition():
    rng = np.random.default_rng(1)
    l, tokens, T = rng.normal(size=(4, 7)), np.array([2, -1, 0, 6]), np.array([1.0, 1.0, 0.5, 2.0])
    g, h = rng.normal(size=4), rng.normal(size=4)

    def f(l):
        lp, H = ref.logprobs(l, tokens, T)
        return (g * lp + h * H).sum()
    np.testing.assert_allclose(ref.gradient(l, tokens, T, g, h), differences(f, l), atol=1e-5)
    assert np.isclose(ref.logprobs(np.zeros((1, 8)), [3])[0][0], -np.log(8)) and np.isclose(ref.logprobs(np.zeros((1, 8)), [3])[1][0], np.log(8))
    lp, H = ref.logprobs(np.array([[-INF] * 3, [0, -INF, -INF], [NAN, 0, 0], [0, INF, 0]]), [0, 0, 0, 0])
    assert lp[0] == -INF and H[0] == 0 and lp[1] == 0 and H[1] == 0 and np.isnan(lp[2:]).all()


def test_loss_definitions():
    # The slopes against differences by the log-probabilities, and a few values by hand.
    rng = np.random.default_rng(2)
    lp, H, old, A, refs = (rng.normal(size=9) for _ in range(5))
    old = lp - np.log(np.array([0.5, 0.7, 0.9, 1.0, 1.1, 1.15, 1.4, 2.0, 1.0]))
    w, live = rng.random(9), np.arange(9) != 4

    def loss(lp, H=H):
        return ref.policy(lp, H, old, A, refs, w, live, 0.2, 0.25, 0.3, 0.1)[0]
    _, kl, clipped, _, slope, hs = ref.policy(lp, H, old, A, refs, w, live, 0.2, 0.25, 0.3, 0.1)
    np.testing.assert_allclose(slope, differences(loss, lp), atol=1e-6)
    np.testing.assert_allclose(hs, differences(lambda H: loss(lp, H), H), atol=1e-6)
    assert kl >= 0
    one = lambda r, a: ref.policy(np.log([r]), np.zeros(1), np.zeros(1), np.array([a]), None, np.ones(1), np.array([True]), 0.2, 0.2, 0, 0)  # noqa: E731
    assert np.isclose(one(2.0, 1.0)[0], -1.2) and one(2.0, 1.0)[4] == 0 and np.isclose(one(2.0, -1.0)[0], 2.0) and one(2.0, 1.0)[2] == 1
    assert np.isclose(one(0.5, 1.0)[0], -0.5) and np.isclose(one(0.5, -1.0)[0], 0.8) and one(0.5, -1.0)[4] == 0 and one(0.5, 1.0)[2] == 0

    tokens, offsets = np.array([1, 1, -1, 1, 1, 1, 1, 1, 1]), np.array([0, 3, 5, 5, 8])
    base = np.where(tokens >= 0, lp, 0)
    base[8] = 0
    for how in (dict(), dict(average=True), dict(smoothing=0.2, margin=0.5)):
        _, d, slope = ref.preference(base, tokens, offsets, refs, 0.7, **how)
        want = differences(lambda v: ref.preference(v, tokens, offsets, refs, 0.7, **how)[0], base)
        np.testing.assert_allclose(slope, np.where(tokens >= 0, want, 0), atol=1e-6)
        assert slope[2] == 0 and slope[8] == 0 and len(d) == 2
    assert np.isclose(ref.preference(np.zeros(9), tokens, offsets, None, 1.0)[0], np.log(2))


# ---- autograd ----------------------------------------------------------------------------------

class StandIn:
    """The native module's calls on CPU tensors (arguments as in csrc/binding.cpp)."""

    def token_logprobs(self, logits, tokens, temperature, entropy, stream):
        lp, H = ref.logprobs(logits.numpy(), tokens.numpy(), temperature)
        f = lambda v: torch.from_numpy(np.asarray(v)).float()  # noqa: E731
        return f(lp), f(H) if entropy else None, torch.zeros(len(lp), 2), temperature

    def token_logprobs_backward(self, logits, tokens, temperature, stats, entropies, g, h, scale, out, stream):
        s = 1.0 if scale is None else scale.item()
        zero = np.zeros(len(tokens))
        return torch.from_numpy(ref.gradient(logits.numpy(), tokens.numpy(), temperature, s * (zero if g is None else g.numpy()),
                                             None if h is None else s * h.numpy())).float()

    def policy_loss(self, logits, tokens, old, A, refs, w, temperature, low, high, kl, entropy, gradient, out, stream):
        lp, H = ref.logprobs(logits.numpy(), tokens.numpy(), temperature)
        got = ref.policy(lp, H, old.numpy(), A.numpy(), None, np.full(len(lp), 1 / len(lp)), np.ones(len(lp), bool), low, high, kl, entropy)
        f = lambda v: torch.from_numpy(np.asarray(v)).float()  # noqa: E731
        return f(got[0]), f(got[1]), f(got[2]), f(got[3]), f(lp), f(H), torch.zeros(len(lp), 2), f(got[4]), f(got[5]), None, temperature

    def preference_loss(self, logits, tokens, offsets, refs, beta, smoothing, margin, average, temperature, stream):
        lp, _ = ref.logprobs(logits.numpy(), tokens.numpy(), temperature)
        loss, d, slopes = ref.preference(lp, tokens.numpy(), offsets.numpy(), None, beta, smoothing, margin, average)
        f = lambda v: torch.from_numpy(np.asarray(v)).float()  # noqa: E731
        return f(loss), f(d), f(lp), torch.zeros(len(lp), 2), f(slopes), temperature


@pytest.fixture()
def losses(pk, monkeypatch):
    from streaming_selection_primitive_gb300 import _lm, _losses
    monkeypatch.setattr(_lm, "_ext", StandIn())
    return _losses


def leaf(rows=6, n=9):
    rng = np.random.default_rng(5)
    return (torch.from_numpy(rng.normal(size=(rows, n)).astype(np.float32)).requires_grad_(), torch.from_numpy(rng.integers(0, n, rows)),
            torch.from_numpy(rng.normal(size=rows).astype(np.float32)))


def calls(losses, z, t, a):
    old = torch.log_softmax(z.detach(), 1)[torch.arange(len(t)), t] - 0.05
    return {"logprobs": lambda: (losses.token_logprobs(z, t).logprobs * a).sum(),
            "entropies": lambda: (losses.token_logprobs(z, t, entropy=True).entropies * a).sum(),
            "policy": lambda: losses.policy_loss(z, t, old, a, entropy=0.1).loss,
            "preference": lambda: losses.preference_loss(z, t, torch.tensor([0, 3, 6])).loss}


@pytest.mark.parametrize("of", ["logprobs", "entropies", "policy", "preference"])
def test_first_and_second_derivative(losses, of):
    z, t, a = leaf()
    call = calls(losses, z, t, a)[of]
    y = call()
    grad, = torch.autograd.grad(y, z, create_graph=True)
    plain, = torch.autograd.grad(call(), z)
    assert torch.equal(grad.detach(), plain) and not plain.requires_grad
    with pytest.raises(NotImplementedError, match="second derivative"):
        (y * 0 + grad.square().sum()).backward()
    twice, = torch.autograd.grad(2 * call(), z)
    torch.testing.assert_close(twice, 2 * plain)


def test_gradients_of_the_plain_formulas(losses):
    z, t, a = leaf()
    got = {of: torch.autograd.grad(call(), z)[0] for of, call in calls(losses, z, t, a).items()}
    rows = torch.arange(6)
    logp = torch.log_softmax(z.double(), 1)
    lp, H = logp[rows, t], -(logp.exp() * logp).sum(1)
    old = torch.log_softmax(z.detach(), 1)[rows, t] - 0.05
    ratio = (lp - old).exp()
    loss = (-torch.minimum(ratio * a, ratio.clamp(0.8, 1.2) * a) - 0.1 * H).mean()
    prefer = -torch.nn.functional.logsigmoid(0.1 * (lp[:3].sum() - lp[3:].sum()))
    for of, y in (("logprobs", (lp * a).sum()), ("entropies", (H * a).sum()), ("policy", loss), ("preference", prefer)):
        want, = torch.autograd.grad(y, z, retain_graph=True)
        torch.testing.assert_close(got[of], want.float(), rtol=1e-5, atol=1e-6)


def test_what_counts_as_a_constant(losses):
    z, t, a = leaf()
    b = a.clone().requires_grad_()
    for call in (lambda: losses.policy_loss(z, t, b, a), lambda: losses.policy_loss(z, t, a, b), lambda: losses.policy_loss(z, t, a, a, ref_logprobs=b),
                 lambda: losses.policy_loss(z, t, a, a, weights=b), lambda: losses.token_logprobs(z, t, temperature=b),
                 lambda: losses.preference_loss(z, t, torch.tensor([0, 3, 6]), ref_logprobs=b)):
        with pytest.raises(ValueError, match="constant"):
            call()
    with pytest.raises(ValueError, match="gradient=True"):
        losses.policy_loss(z, t, a, a, out=torch.empty_like(z))
    with torch.no_grad():
        assert not losses.token_logprobs(z, t).logprobs.requires_grad
    r = losses.token_logprobs(z, t, entropy=True)
    assert torch.autograd.grad(r.logprobs.sum(), z, retain_graph=True)[0] is not None  # without the entropies' part
    with pytest.raises(ValueError, match="hidden states"):
        losses.token_logprobs_backward(z, t, r._replace(stats=None))
