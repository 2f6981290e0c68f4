"""The selections of a language model: a token from logits, the experts of a token.

    tokens, logprobs = pk.sample_tokens(logits, noise, temperature=0.8, top_k=50, top_p=0.9)
    r = pk.route(router_logits, k=8)               # r.gates, r.experts, r.counts, r.loss
    dz = pk.route_backward(router_logits, r, grad_gates=dg, grad_loss=dl)

As in the rest of the package, everything runs in the library's kernels on the
current stream (or ``stream``), and a tensor that the kernels cannot read as
it is raises instead of being copied.  A call given ``stream`` marks the
outputs that it makes as used there; the inputs' lifetime is the caller's.
"""
from __future__ import annotations

import ctypes as C
from typing import Any, NamedTuple

from . import _abi

_types = {}  # torch dtype -> profk_type


def _torch():
    import torch
    if not _types:
        _types.update({torch.float32: _abi.F32, torch.bfloat16: _abi.BF16, torch.float16: _abi.F16})
    return torch


def _stream_of(torch, stream, device) -> int:
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _logits(torch, x):
    """(rows, columns, row stride, type) of a 2-D CUDA tensor of logits."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in _types:
        raise TypeError("logits must be a float32, bfloat16 or float16 CUDA tensor")
    if x.dim() != 2:
        raise ValueError("logits must be 2-D")
    rows, n = x.shape
    if n > 1 and x.stride(1) != 1:
        raise ValueError("logits must have unit column stride")
    return rows, n, (x.stride(0) if rows > 1 else n), _types[x.dtype]


def _array(torch, t, name, shape, dtype, device):
    """Checks a contiguous CUDA tensor and returns its address."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        raise TypeError(f"{name} must be a {str(dtype)[6:]} tensor on {device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {tuple(shape)}")
    return t.data_ptr()


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
    inputs give the same token and log-probability."""
    torch = _torch()
    rows, n, ld, kind = _logits(torch, logits)
    device = logits.device
    if not isinstance(noise, torch.Tensor) or noise.dtype != torch.float32 or noise.device != device:
        raise TypeError(f"noise must be a float32 tensor on {device}")
    if noise.shape != logits.shape or (n > 1 and noise.stride(1) != 1):
        raise ValueError("noise must have the logits' shape and unit column stride")
    how = _abi.Sampling()
    per_row = (rows,)
    if isinstance(temperature, torch.Tensor):
        how.temperature = _array(torch, temperature, "temperature", per_row, torch.float32, device)
    else:
        how.all_temperature = temperature
    if isinstance(top_k, torch.Tensor):
        how.top_k = _array(torch, top_k, "top_k", per_row, torch.int32, device)
    else:
        how.all_top_k = min(max(int(top_k), 0), 2**31 - 1)
    if isinstance(top_p, torch.Tensor):
        how.top_p = _array(torch, top_p, "top_p", per_row, torch.float32, device)
    else:
        how.all_top_p = top_p
    if isinstance(min_p, torch.Tensor):
        how.min_p = _array(torch, min_p, "min_p", per_row, torch.float32, device)
    else:
        how.all_min_p = min_p
    mask_ptr, mask_ld = None, 0
    if mask is not None:
        words = (n + 31) // 32
        if not isinstance(mask, torch.Tensor) or mask.dtype != torch.int32 or mask.device != device:
            raise TypeError(f"mask must be an int32 tensor on {device}")
        if mask.shape != (rows, words) or (words > 1 and mask.stride(1) != 1):
            raise ValueError(f"mask must have shape {(rows, words)} and unit column stride")
        mask_ptr, mask_ld = mask.data_ptr(), (mask.stride(0) if rows > 1 else words)
    if out is None:
        tokens = torch.empty(rows, dtype=torch.int64, device=device)
        logprobs = torch.empty(rows, dtype=torch.float32, device=device)
        if stream is not None:
            tokens.record_stream(stream)
            logprobs.record_stream(stream)
        tp, lp = tokens.data_ptr(), logprobs.data_ptr()
    else:
        tokens, logprobs = out
        tp = _array(torch, tokens, "out[0]", per_row, torch.int64, device)
        lp = _array(torch, logprobs, "out[1]", per_row, torch.float32, device)
    code = _abi.lib().profk_sample_tokens(logits.data_ptr(), kind, rows, n, ld, noise.data_ptr(),
                                          noise.stride(0) if rows > 1 else n, mask_ptr, mask_ld, how, tp, lp,
                                          _stream_of(torch, stream, device))
    if code:
        _abi.check(code)
    return tokens, logprobs


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


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    return _SCORES[score]


def route(logits, k: int, *, score: str = "softmax", normalize: bool = True, bias=None, mask=None, balance: bool = True,
          stream=None) -> Routing:
    """Top-k experts of each token with their gates, the count of tokens per
    expert and, with ``balance``, the balance loss (1 for an even choice).

    logits: (tokens, experts), float32, bfloat16 or float16, unit column
    stride, at most 1024 experts.  k: at most 32.  score "softmax": gates from
    the softmax of the logits; "sigmoid": from their sigmoids.  normalize: a
    token's gates sum to 1.  bias: (experts,) float32, added to the logits for
    the choice only.  mask: (tokens,) bool, False where a token is not routed:
    its slots hold expert -1 and gate 0.  A -inf logit is never chosen.  Equal
    values are chosen by lower index.

    Where logits requires a gradient, gates and loss carry it (route_backward)."""
    torch = _torch()
    if torch.is_grad_enabled() and isinstance(logits, torch.Tensor) and logits.requires_grad:
        if stream is not None:
            raise ValueError("a call that records a gradient runs on the current stream: use torch.cuda.stream")
        gates, experts, counts, loss = _autograd(torch).apply(logits, k, score, normalize, bias, mask, balance)
        return Routing(gates, experts, counts, loss, score, normalize)
    tokens, E, ld, kind = _logits(torch, logits)
    device = logits.device
    how = _abi.Routing(_score(score), 1 if normalize else 0)
    if bias is not None:
        how.bias = _array(torch, bias, "bias", (E,), torch.float32, device)
    if mask is not None:
        how.mask = _array(torch, mask, "mask", (tokens,), torch.bool, device)
    k = int(k)
    if k < 1 or k > E:
        raise ValueError("k must be in 1 .. experts")
    gates = torch.empty((tokens, k), dtype=torch.float32, device=device)
    experts = torch.empty((tokens, k), dtype=torch.int64, device=device)
    counts = torch.empty(E, dtype=torch.int64, device=device)
    loss = torch.empty((), dtype=torch.float32, device=device) if balance else None
    if stream is not None:
        for t in (gates, experts, counts) + ((loss,) if balance else ()):
            t.record_stream(stream)
    code = _abi.lib().profk_route(logits.data_ptr(), kind, tokens, E, ld, k, how, gates.data_ptr(), experts.data_ptr(),
                                  counts.data_ptr(), loss.data_ptr() if balance else None,
                                  _stream_of(torch, stream, device))
    if code:
        _abi.check(code)
    return Routing(gates, experts, counts, loss, score, normalize)


def route_backward(logits, routing: Routing, *, grad_gates=None, grad_loss=None, out=None, stream=None):
    """Gradient of route()'s gates and loss with respect to the logits, in the
    logits' type; the choice and the counts are constants.

    grad_gates: (tokens, k) float32, or None.  grad_loss: a float32 tensor of one
    element on the device, or None.  routing.counts may have been replaced by
    the sum over several devices.  out: where to write, unit column stride."""
    torch = _torch()
    tokens, E, ld, kind = _logits(torch, logits)
    device = logits.device
    if routing.experts.dim() != 2:
        raise ValueError("routing.experts must be 2-D")
    k = routing.experts.shape[1]
    chosen = _array(torch, routing.experts, "routing.experts", (tokens, k), torch.int64, device)
    how = _abi.Routing(_score(routing.score), 1 if routing.normalize else 0)
    gg = gl = counts = None
    if grad_gates is not None:
        gg = _array(torch, grad_gates, "grad_gates", (tokens, k), torch.float32, device)
    if grad_loss is not None:
        if grad_loss.numel() != 1:
            raise ValueError("grad_loss must hold one element")
        gl = _array(torch, grad_loss, "grad_loss", grad_loss.shape, torch.float32, device)
        counts = _array(torch, routing.counts, "routing.counts", (E,), torch.int64, device)
    if out is None:
        out = torch.empty((tokens, E), dtype=logits.dtype, device=device)
        if stream is not None:
            out.record_stream(stream)
        out_ld = E
    else:
        if not isinstance(out, torch.Tensor) or out.dtype != logits.dtype or out.device != device:
            raise TypeError("out must have the logits' type and device")
        if out.shape != logits.shape or (E > 1 and out.stride(1) != 1):
            raise ValueError("out must have the logits' shape and unit column stride")
        out_ld = out.stride(0) if tokens > 1 else E
    code = _abi.lib().profk_route_backward(logits.data_ptr(), kind, tokens, E, ld, k, how, chosen, counts, gg, gl,
                                           out.data_ptr(), out_ld, _stream_of(torch, stream, device))
    if code:
        _abi.check(code)
    return out


_function = None


def _autograd(torch):
    """The autograd function behind route(), made on first use (torch is imported lazily)."""
    global _function
    if _function is None:
        class Route(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, k, score, normalize, bias, mask, balance):
                r = route(logits.detach(), k, score=score, normalize=normalize, bias=bias, mask=mask, balance=balance)
                ctx.save_for_backward(logits, r.experts, r.counts)
                ctx.how = score, normalize
                ctx.mark_non_differentiable(r.experts, r.counts)
                ctx.set_materialize_grads(False)
                return r.gates, r.experts, r.counts, r.loss

            @staticmethod
            def backward(ctx, grad_gates, _experts, _counts, grad_loss):
                logits, experts, counts = ctx.saved_tensors
                r = Routing(None, experts, counts, None, *ctx.how)
                if grad_gates is not None:
                    grad_gates = grad_gates.float().contiguous()
                if grad_loss is not None:
                    grad_loss = grad_loss.float().contiguous()
                grad = route_backward(logits.detach(), r, grad_gates=grad_gates, grad_loss=grad_loss)
                return (grad,) + (None,) * 6
        _function = Route
    return _function
