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
