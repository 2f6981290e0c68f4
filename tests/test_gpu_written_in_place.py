"""Tensors that a call is given to write to: autograd notices, as of torch's own operations."""
import pytest
import torch

from logprob_checks import make

pytestmark = pytest.mark.gpu


def setting(dtype=torch.float32):
    z, t, _ = make(12, 40, dtype)
    one = torch.ones(12, device=z.device)
    return z, t, one, torch.tensor([0, 6, 12], device=z.device)


def recorded(pk, x, t, one, o):
    return {"logprobs": lambda: pk.token_logprobs(x, t).logprobs.sum(), "policy": lambda: pk.policy_loss(x, t, -4 * one, one).loss,
            "preference": lambda: pk.preference_loss(x, t, o).loss}


def writers(pk, z, t, one, o):
    r, p, q = pk.token_logprobs(z, t), pk.policy_loss(z, t, -4 * one, one), pk.preference_loss(z, t, o)
    return {"logprobs": lambda x, out: pk.token_logprobs_backward(x, t, r, grad_logprobs=one, out=out),
            "policy": lambda x, out: pk.policy_loss_backward(x, t, p, out=out),
            "preference": lambda x, out: pk.preference_loss_backward(x, t, q, out=out),
            "with the loss": lambda x, out: pk.policy_loss(x, t, -4 * one, one, gradient=True, out=out).grad_logits}


@pytest.mark.parametrize("of", ["logprobs", "policy", "preference"])
@pytest.mark.parametrize("writer", ["logprobs", "policy", "preference", "with the loss"])
def test_logits_that_a_recorded_call_has_saved(pk, cuda_device, of, writer):
    z, t, one, o = setting()
    write = writers(pk, z, t, one, o)[writer]
    leaf = z.clone().requires_grad_()
    want = torch.autograd.grad(recorded(pk, leaf, t, one, o)[of](), leaf)[0]
    for place in (lambda x: x, lambda x: x.detach(), lambda x: x[:], lambda x: x.view(12, 40)):
        x = leaf * 1.0
        y = recorded(pk, x, t, one, o)[of]()
        got = write(x.detach(), place(x))
        assert got.data_ptr() == x.data_ptr() and not torch.equal(x, z)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    x = leaf * 1.0  # written elsewhere: nothing to notice
    y = recorded(pk, x, t, one, o)[of]()
    write(x.detach(), torch.empty_like(z))
    assert torch.equal(torch.autograd.grad(y, leaf)[0], want)


def test_what_torch_has_saved(pk, cuda_device):
    z, t, one, o = setting()
    for write in writers(pk, z, t, one, o).values():
        leaf = z.clone().requires_grad_()
        x = torch.tanh(leaf)  # saved as its result
        write(x.detach(), x)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            x.sum().backward()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_gradient_over_logits_that_a_product_made(pk, cuda_device, dtype):
    # The product has not saved its result: its gradient can take the logits' memory.
    z, t, one, o = setting()
    hidden = torch.randn(12, 16, device=cuda_device).to(dtype)
    weight = torch.randn(40, 16, device=cuda_device).to(dtype).requires_grad_()
    plain = pk.policy_loss((hidden @ weight.t()).detach(), t, -4 * one, one, gradient=True).grad_logits
    logits = hidden @ weight.t()
    r = pk.policy_loss(logits, t, -4 * one, one, gradient=True, out=logits)
    logits.backward(r.grad_logits)
    want, = torch.autograd.grad(hidden @ weight.t(), weight, plain)
    assert torch.equal(weight.grad, want) and torch.equal(r.grad_logits, plain)


def test_leaves(pk, cuda_device):
    z, t, one, o = setting()
    for write in writers(pk, z, t, one, o).values():
        leaf = z.clone().requires_grad_()
        for out in (leaf, leaf[:], leaf.view(12, 40)):
            with pytest.raises(ValueError, match="leaf"):
                write(z, out)
        assert torch.equal(leaf, z) and leaf._version == 0
        got = write(z, torch.empty_like(z))
        with torch.no_grad():
            assert torch.equal(write(z, leaf), got) and torch.equal(leaf, got)
        assert leaf._version == 1
        assert torch.equal(write(z, leaf.detach()), got) and leaf._version == 2


def test_versions(pk, cuda_device):
    z, t, one, o = setting()
    for write in writers(pk, z, t, one, o).values():
        out, before = torch.empty_like(z), z._version
        write(z, out)
        assert out._version == 1 and z._version == before
        both = torch.zeros(24, 40, device=cuda_device)
        with pytest.raises(pk.ProfkError):  # across the logits: refused, so nothing is written
            write(both[:12], both[1:13])
        assert both._version == 0
        with torch.inference_mode():
            inner = torch.empty_like(z)
            write(z, inner)
        write(z, inner)
        assert torch.equal(inner, out)


def test_the_selections_outputs(pk, cuda_device):
    z, t, one, o = setting()
    noise = torch.empty_like(z).exponential_()
    out = (torch.empty(12, dtype=torch.int64, device=cuda_device), torch.empty(12, device=cuda_device))
    pk.sample_tokens(z, noise, out=out)
    assert [v._version for v in out] == [1, 1]
    r = pk.route(z, 4)
    place = torch.empty_like(z)
    pk.route_backward(z, r, grad_gates=torch.ones(12, 4, device=cuda_device), out=place)
    assert place._version == 1
    leaf = torch.randn(50, 8, device=cuda_device, requires_grad=True)
    tokens = torch.zeros(12, dtype=torch.int64, device=cuda_device)
    y = leaf[tokens].square().sum()  # saves the index
    pk.sample_tokens(z, noise, out=(tokens, out[1]))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
