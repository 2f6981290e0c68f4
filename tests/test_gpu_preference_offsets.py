"""Preference loss: offsets that fall or leave the rows make everything NaN that they could have a say in, the same each time."""
import pytest
import torch

from logprob_checks import make

pytestmark = pytest.mark.gpu


def bad_offsets(pairs, rows):
    even = torch.linspace(0, rows, 2 * pairs + 1).long()
    for at, value in ((0, -1), (2 * pairs, rows + 1), (1, rows + 1), (2 * pairs - 1, -1), (pairs, 1 << 40), (pairs, -(1 << 62)), (0, 1 << 62)):
        o = even.clone()
        o[at] = value
        yield o
    o = even.clone()  # two sequences, each in order by itself, that share rows
    o[pairs] = o[max(pairs - 2, 0)]
    o[pairs - 1] = o[pairs] + 3
    yield o
    yield even.flip(0)


@pytest.mark.parametrize("pairs,rows", [(1, 20), (2, 20), (3, 700), (20, 300), (600, 3000)])
@pytest.mark.parametrize("average", [False, True])
def test_bad_offsets(pk, cuda_device, pairs, rows, average):
    logits, tokens, _ = make(rows, 100, torch.float32, left_out=0.2)
    sound = torch.linspace(0, rows, 2 * pairs + 1).long().to(cuda_device)
    want = pk.preference_loss(logits, tokens, sound, average=average)
    row = torch.arange(rows, device=cuda_device)
    for bad in bad_offsets(pairs, rows):
        if (bad[1:] >= bad[:-1]).all() and bad[0] >= 0 and bad[-1] <= rows:
            continue  # (few pairs: not all of the changes make them bad)
        r = pk.preference_loss(logits, tokens, bad.to(cuda_device), average=average)
        live = (tokens >= 0) & (row >= bad[0].item()) & (row < bad[-1].item())
        assert r.loss.isnan() and r.margins.isnan().all() and r.margins.shape == (pairs,)
        assert r.slopes[live].isnan().all() and (r.slopes[~live] == 0).all()
        grad = pk.preference_loss_backward(logits, tokens, r)
        assert grad[live].isnan().all() and (grad[~live] == 0).all()
    again = pk.preference_loss(logits, tokens, sound, average=average)
    assert all(torch.equal(a, b) for a, b in zip(want[:5], again[:5])) and not want.loss.isnan()


def test_no_pair_needs_no_offsets(pk, cuda_device):
    logits, tokens, _ = make(20, 100, torch.float32)
    for first in (-5, 0, 30):
        r = pk.preference_loss(logits, tokens, torch.tensor([first], device=cuda_device))
        assert r.loss == 0 and (r.slopes == 0).all() and (r.logprobs == 0).all()
    none = pk.preference_loss(logits[:0], tokens[:0], torch.tensor([0, 0, 0], device=cuda_device))
    assert none.margins.tolist() == [0.0]
    bad = pk.preference_loss(logits[:0], tokens[:0], torch.tensor([0, 1, 0], device=cuda_device))
    assert bad.loss.isnan() and bad.margins.isnan().all()


def test_bad_offsets_under_autograd_and_in_a_graph(pk, cuda_device):
    logits, tokens, _ = make(20, 100, torch.float32)
    offsets = torch.tensor([0, 5, 10, 15, 20], device=cuda_device)
    leaf = logits.clone().requires_grad_()
    pk.preference_loss(leaf, tokens, torch.tensor([0, 5, 3, 8, 20], device=cuda_device)).loss.backward()
    assert leaf.grad.isnan().all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = pk.preference_loss(logits, tokens, offsets)
    want = pk.preference_loss(logits, tokens, offsets)
    for bad in (True, False, True, False):  # what was bad is not kept
        offsets[2] = 4 if bad else 10
        graph.replay()
        assert r.margins.isnan().all() and r.slopes.isnan().all() if bad else torch.equal(r.margins, want.margins) and torch.equal(r.slopes, want.slopes)
