"""The selections of a language model: a token from logits, the experts of a token.

    tokens, logprobs = pk.sample_tokens(logits, noise, temperature=0.8, top_k=50, top_p=0.9)
    r = pk.route(router_logits, k=8)               # r.gates, r.experts, r.counts, r.loss
    dz = pk.route_backward(router_logits, r, grad_gates=dg, grad_loss=dl)

As in the rest of the package, everything runs in the library's kernels on the
current stream (or ``stream``), and a tensor that the kernels cannot read as
it is raises instead of being copied.  A call given ``stream`` makes its outputs
on that stream, so that it waits for nothing on the current one, and marks them as
used on the current stream as well; the caller orders the two where they meet, and
the inputs' lifetime is the caller's.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
from typing import Any, NamedTuple

from . import _abi

_ext = None


def _native():
    """The module built from csrc/binding.cpp (for the installed torch); raises if it is missing."""
    global _ext
    if _ext is None:
        from .build import binding_path
        path = binding_path()
        if not path.exists():
            raise ImportError(f"{path} is missing: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        _abi.lib()
        loader = importlib.machinery.ExtensionFileLoader("profk_torch", str(path))
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("profk_torch", loader))
        loader.exec_module(ext)
        _ext = ext
    return _ext


def sample_tokens(logits, noise, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mask=None, out=None, stream=None):
    """One token per row of logits: (tokens int64, logprobs float32).

    logits: 2-D, float32, bfloat16 or float16, unit column stride.  noise: float32
    of the same shape, independent Exp(1) numbers (``Tensor.exponential_``);
    rows may share memory (``expand``).  temperature, top_k, top_p and min_p: a
    number for every row, or a tensor of one per row (float32; top_k int32).
    mask: int32, (rows, ceil(n / 32)), bit i % 32 of word i // 32 set where
    token i is allowed.  The filters are applied in that order, each to what the
    one before kept; temperature 0 takes the largest logit.  A row with nothing
    to choose gives (-1, -inf), one with an allowed NaN (-1, nan).  The same
    inputs give the same token and log-probability.

    Not differentiable: the log-probabilities come without a graph, also where
    logits or temperature require a gradient (what of either has a forward-mode
    tangent raises).  For a loss take them anew from the logits."""
    r = (_ext or _native()).sample_tokens(logits, noise, temperature, top_k, top_p, min_p, mask, out,
                                          None if stream is None else stream.cuda_stream)
    if type(r) is int:
        _abi.check(r)
    return r


class Routing(NamedTuple):
    """What route() returns: gates (tokens, k) float32, experts (tokens, k) int64
    (-1: an empty slot), counts (experts,) int64, loss (a float32 scalar tensor,
    or None), and the score and normalize that it was called with."""
    gates: Any
    experts: Any
    counts: Any
    loss: Any
    score: str
    normalize: bool


_SCORES = {"softmax": _abi.SCORE_SOFTMAX, "sigmoid": _abi.SCORE_SIGMOID}
_BIAS_ON = {"logits": 0, "scores": _abi.BIAS_ON_SCORES}


def _torch():
    import torch
    return torch


def route(logits, k: int, *, score: str = "softmax", normalize: bool = True, bias=None, mask=None, balance: bool = True,
          bias_on: str = "logits", stream=None) -> Routing:
    """Top-k experts of each token with their gates, the count of tokens per
    expert and, with ``balance``, the balance loss (1 for an even choice).

    logits: (tokens, experts), float32, bfloat16 or float16, unit column
    stride, at most 1024 experts.  k: at most 32.  score "softmax": gates from
    the softmax of the logits; "sigmoid": from their sigmoids.  normalize: a
    token's gates sum to 1.  bias: (experts,) float32, for the choice only.
    bias_on "logits": the choice is by z + bias; "scores": by sigmoid(z) + bias or
    softmax(z) + bias, another order (balancing rules that correct a bias step
    by step are mostly stated so, for sigmoid scores above all).  mask: (tokens,) bool, False where a token is not routed:
    its slots hold expert -1 and gate 0.  A -inf logit is never chosen.  Equal
    values are chosen by lower index.

    Where logits requires a gradient, gates and loss carry it (route_backward).
    There is no second derivative: going back through a gradient that was taken
    with create_graph raises.  Nor is there one in forward mode: logits with a
    tangent raise."""
    code = _SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    on = _BIAS_ON.get(bias_on)
    if on is None:
        raise ValueError(f"bias_on must be one of {sorted(_BIAS_ON)}")
    if getattr(logits, "requires_grad", False) and _torch().is_grad_enabled():
        if stream is not None:
            raise ValueError("a call that records a gradient runs on the current stream: use torch.cuda.stream")
        return Routing(*_autograd().apply(logits, k, score, normalize, bias, mask, balance, bias_on), score, normalize)
    r = (_ext or _native()).route(logits, k, code + on, bool(normalize), bias, mask, bool(balance),
                                  None if stream is None else stream.cuda_stream)
    if type(r) is int:
        _abi.check(r)
    return Routing(*r, score, normalize)


def route_backward(logits, routing: Routing, *, grad_gates=None, grad_loss=None, out=None, stream=None):
    """Gradient of route()'s gates and loss with respect to the logits, in the
    logits' type; the choice and the counts are constants.

    grad_gates: (tokens, k) float32, or None.  grad_loss: a float32 tensor of one
    element on the device, or None.  routing.counts may have been replaced by
    the sum over several devices.  out: where to write, unit column stride.
    The result comes without a graph; a forward-mode tangent raises."""
    code = _SCORES.get(routing.score)
    if code is None:
        raise ValueError(f"routing.score must be one of {sorted(_SCORES)}")
    r = (_ext or _native()).route_backward(logits, routing.experts, routing.counts, code, bool(routing.normalize),
                                           grad_gates, grad_loss, out, None if stream is None else stream.cuda_stream)
    if type(r) is int:
        _abi.check(r)
    return r


_function = None


def _autograd():
    """The autograd function behind route(), made on first use (torch is imported lazily)."""
    global _function
    if _function is None:
        torch = _torch()

        def gradient(logits, experts, counts, grad_gates, grad_loss, score, normalize):
            r = Routing(None, experts, counts, None, score, normalize)
            if grad_gates is not None:
                grad_gates = grad_gates.detach().float().contiguous()
            if grad_loss is not None:
                grad_loss = grad_loss.detach().float().contiguous()
            return route_backward(logits.detach(), r, grad_gates=grad_gates, grad_loss=grad_loss)

        class Route(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, k, score, normalize, bias, mask, balance, bias_on):
                r = route(logits.detach(), k, score=score, normalize=normalize, bias=bias, mask=mask, balance=balance,
                          bias_on=bias_on)
                ctx.save_for_backward(logits, r.experts, r.counts)
                ctx.how = score, normalize
                ctx.mark_non_differentiable(r.experts, r.counts)
                ctx.set_materialize_grads(False)
                return r.gates, r.experts, r.counts, r.loss

            @staticmethod
            def backward(ctx, grad_gates, _experts, _counts, grad_loss):
                of = RouteGradient.apply if torch.is_grad_enabled() else gradient
                return (of(*ctx.saved_tensors, grad_gates, grad_loss, *ctx.how),) + (None,) * 7

        class RouteGradient(torch.autograd.Function):
            """The gradient under create_graph: what is made of it leads back here, to the logits and to the
            gradients of gates and loss, instead of counting as a constant."""

            @staticmethod
            def forward(ctx, *args):
                return gradient(*args)

            @staticmethod
            def backward(ctx, _grad):
                raise NotImplementedError("route has no second derivative")
        _function = Route
    return _function
