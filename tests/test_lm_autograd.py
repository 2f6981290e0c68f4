"""route's place in autograd, without a GPU: the native half is replaced by the definitions in float64."""
import numpy as np
import pytest
import torch

from oracle import selections as ref


class StandIn:
    """The native module's calls on CPU tensors (arguments as in csrc/binding.cpp)."""

    NAMES = {0: "softmax", 1: "sigmoid"}

    def route(self, logits, k, score, normalize, bias, mask, balance, stream):
        gates, experts, counts, loss = ref.routing(logits.numpy(), k, self.NAMES[score], normalize)
        return (torch.from_numpy(gates).float(), torch.from_numpy(experts), torch.from_numpy(counts),
                torch.tensor(loss, dtype=torch.float32) if balance else None)

    def route_backward(self, logits, experts, counts, score, normalize, grad_gates, grad_loss, out, stream):
        return torch.from_numpy(ref.routing_gradient(
            logits.numpy(), experts.numpy(), counts.numpy(), self.NAMES[score], normalize,
            None if grad_gates is None else grad_gates.numpy(), None if grad_loss is None else grad_loss.item())).float()


@pytest.fixture()
def lm(pk, monkeypatch):
    from streaming_selection_primitive_gb300 import _lm
    monkeypatch.setattr(_lm, "_ext", StandIn())
    return _lm


def leaf(tokens=6, experts=9):
    return torch.from_numpy(np.random.default_rng(5).normal(size=(tokens, experts)).astype(np.float32)).requires_grad_()


@pytest.mark.parametrize("of", ["gates", "loss"])
def test_a_second_derivative_raises(lm, of):
    # What is made of the first gradient depends on the logits: a penalty on it must not count as a constant,
    # also where the gradient that came in (here of a plain sum) requires none.
    z = leaf()
    r = lm.route(z, 3, normalize=False)
    y = r.gates.sum() if of == "gates" else r.loss
    grad, = torch.autograd.grad(y, z, create_graph=True)
    plain, = torch.autograd.grad(lm.route(z, 3, normalize=False)._asdict()[of].sum(), z)
    assert torch.equal(grad.detach(), plain) and not plain.requires_grad
    with pytest.raises(NotImplementedError):
        (y * 0 + grad.square().sum()).backward()


def test_a_graph_that_is_not_gone_through_does_not_raise(lm):
    z = leaf()
    r = lm.route(z, 3)
    weight = torch.ones(r.gates.shape, requires_grad=True)
    (r.gates * weight).sum().backward(create_graph=True)
    first, z.grad = z.grad, None
    (lm.route(z, 3).gates * weight.detach()).sum().backward()
    assert torch.equal(first.detach(), z.grad) and torch.equal(weight.grad.detach(), r.gates.detach())


def test_first_derivative_of_gates_and_loss(lm):
    z = leaf()
    r = lm.route(z, 2, score="sigmoid")
    dg = torch.linspace(-1, 1, r.gates.numel()).view_as(r.gates)
    ((r.gates * dg).sum() + 3 * r.loss).backward()
    want = ref.routing_gradient(z.detach().numpy(), r.experts.numpy(), r.counts.numpy(), "sigmoid", True, dg.numpy(), 3.0)
    np.testing.assert_allclose(z.grad.numpy(), want, rtol=0, atol=1e-6)
    with torch.no_grad():
        assert not lm.route(z, 2).gates.requires_grad


def test_what_a_bias_is_added_to(pk, lm, monkeypatch):
    # The code that reaches the native half, and the C-ABI's refusal of other ones.
    import ctypes as C

    from streaming_selection_primitive_gb300 import _abi
    seen = []
    real = StandIn.route
    monkeypatch.setattr(StandIn, "route", lambda self, logits, k, score, *rest: (seen.append(score), real(self, logits, k, score & 1, *rest))[1])
    for score in ("softmax", "sigmoid"):
        for on in ("logits", "scores"):
            lm.route(leaf().detach(), 2, score=score, bias_on=on)
            lm.route(leaf(), 2, score=score, bias_on=on)
    assert seen == [0, 0, 0x100, 0x100, 1, 1, 0x101, 0x101]
    with pytest.raises(ValueError):
        lm.route(leaf(), 2, bias_on="gates")
    p = C.c_void_p(256)
    for code in (2, 0x102, 0x200, 0x201, -1):
        how = _abi.Routing(code, 1)
        assert pk.lib().profk_route(p, _abi.F32, 4, 16, 16, 2, how, p, p, p, None, None) == _abi.PROFK_ERR_INVALID
        assert pk.lib().profk_route_backward(p, _abi.F32, 0, 16, 16, 2, how, p, p, p, None, p, 16, None) == _abi.PROFK_ERR_INVALID
    assert pk.lib().profk_route_backward(p, _abi.F32, 0, 16, 16, 2, _abi.Routing(0x101, 1), p, p, p, None, p, 16, None) == 0
