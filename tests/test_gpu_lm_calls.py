"""How the language-model selections are called: derivatives, streams, host threads, messages."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

pytestmark = pytest.mark.gpu


def rows(device, tokens=10, experts=16, seed=1):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randn((tokens, experts), generator=g, device=device), g


def test_forward_mode_is_refused(pk, cuda_device):
    z, g = rows(cuda_device)
    noise = torch.empty_like(z).exponential_(generator=g)
    one = torch.ones(10, device=cuda_device)
    r = pk.route(z, 2)
    dg, dl = torch.ones_like(r.gates), torch.ones((), device=cuda_device)
    with fwd.dual_level():
        dual = lambda t: fwd.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: pk.route(dual(z), 2), lambda: pk.sample_tokens(dual(z), noise),
                     lambda: pk.sample_tokens(z, noise, temperature=dual(one)),
                     lambda: pk.route_backward(dual(z), r, grad_gates=dg),
                     lambda: pk.route_backward(z, r, grad_gates=dual(dg)),
                     lambda: pk.route_backward(z, r, grad_gates=dg, grad_loss=dual(dl))):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        with pytest.raises(RuntimeError):
            pk.route(dual(z.clone().requires_grad_()), 2)
        # The choice does not vary with the noise or the bias, nor do the outputs.
        pk.sample_tokens(z, dual(noise))
        pk.route(z, 2, bias=dual(torch.ones(16, device=cuda_device)))
    assert torch.equal(pk.route(z, 2).gates, r.gates)


def test_function_transforms_are_refused(pk, cuda_device):
    z, g = rows(cuda_device)
    with pytest.raises(Exception):
        torch.func.jvp(lambda t: pk.route(t, 2).gates, (z,), (torch.ones_like(z),))
    with pytest.raises(Exception):
        torch.func.grad(lambda t: pk.route(t, 2).gates.square().sum())(z)
    with pytest.raises(Exception):
        torch.vmap(lambda t: pk.route(t, 2).gates)(z.expand(3, 10, 16))
    with pytest.raises(Exception):
        torch.vmap(lambda t: pk.sample_tokens(t, torch.ones_like(z))[0])(z.expand(3, 10, 16))


@pytest.mark.parametrize("of", ["gates", "loss"])
def test_a_second_derivative_raises(pk, cuda_device, of):
    z, _ = rows(cuda_device)
    z.requires_grad_()
    r = pk.route(z, 2, normalize=False)
    y = r.gates.sum() if of == "gates" else r.loss
    grad, = torch.autograd.grad(y, z, create_graph=True)
    with pytest.raises(NotImplementedError):
        (y * 0 + grad.square().sum()).backward()


def test_log_probabilities_come_without_a_graph(pk, cuda_device):
    z, g = rows(cuda_device)
    noise = torch.empty_like(z).exponential_(generator=g)
    want = pk.sample_tokens(z, noise)
    got = pk.sample_tokens(z.clone().requires_grad_(), noise)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not got[1].requires_grad
