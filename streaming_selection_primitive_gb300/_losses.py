"""Log-probabilities of given tokens, and the losses that train on them.

    r = pk.token_logprobs(logits, tokens, entropy=True)       # r.logprobs, r.entropies; differentiable
    r = pk.token_logprobs(hidden, tokens, weight=head)        # without the logits ever being in memory
    r = pk.policy_loss(logits, tokens, old, advantages, ref_logprobs=ref, kl=0.05)      # r.loss, r.kl, r.clipped
    r = pk.preference_loss(logits, tokens, offsets, ref_logprobs=ref, beta=0.1)         # r.loss, r.margins

Where logits requires a gradient, what these give carries it; without autograd the `_backward` calls
give it, and policy_loss(..., gradient=True) gives it with the loss.  What holds for _lm.py (streams, no
copies, no forward-mode or second derivatives) holds here.
"""
from __future__ import annotations

from typing import Any, NamedTuple

from . import _abi, _lm
from ._lm import _torch


def _ext():
    """The native half.  Its calls return their outputs and the temperature, or a status."""
    return _lm._ext or _lm._native()


def _made(kind, r):
    """The outputs as a named tuple (made without its constructor, a Python function); a status raises."""
    if type(r) is int:
        _abi.check(r)
    return tuple.__new__(kind, r) if kind else r


def _handle(stream):
    return None if stream is None else stream.cuda_stream


class TokenLogprobs(NamedTuple):
    """What token_logprobs() returns: logprobs (rows,) float32, entropies (rows,) float32 or None, stats
    (rows, 2) float32 (a row's largest logit, and the sum of exp((l - largest) / T); None from hidden states),
    and the temperature that it was called with."""
    logprobs: Any
    entropies: Any
    stats: Any
    temperature: Any


class PolicyLoss(NamedTuple):
    """What policy_loss() returns: loss, kl (the weighted sum of the KL terms, before their factor; 0 without a
    reference), clipped (the weight of the tokens whose ratio is clipped) and entropy (the weighted sum of the
    entropies; 0 where they were not asked for), float32 scalar tensors; logprobs (rows,) float32; entropies
    (rows,) float32 or None; stats and slopes (rows: d loss / d logprob), entropy_slopes (or None), for
    policy_loss_backward; grad_logits (or None); the temperature."""
    loss: Any
    kl: Any
    clipped: Any
    entropy: Any
    logprobs: Any
    entropies: Any
    stats: Any
    slopes: Any
    entropy_slopes: Any
    grad_logits: Any
    temperature: Any


class PreferenceLoss(NamedTuple):
    """What preference_loss() returns: loss, a float32 scalar tensor; margins (pairs,) float32; logprobs (rows,)
    float32; stats and slopes (rows: d loss / d logprob) for preference_loss_backward; the temperature."""
    loss: Any
    margins: Any
    logprobs: Any
    stats: Any
    slopes: Any
    temperature: Any


def token_logprobs(x, tokens, *, weight=None, temperature=1.0, entropy: bool = False, stream=None) -> TokenLogprobs:
    """The log-probability of one given token per row and, with `entropy`, the row's entropy: of the softmax of
    the logits at a temperature.

    x: logits, (rows, n), float32, bfloat16 or float16, unit column stride.  Or, with
    `weight` (n, width), hidden states (rows, width), both bfloat16 or both float16, of 16-byte aligned rows:
    the logits are then their product x @ weight.T in float32, which is never in memory; width may be odd.
    tokens: (rows,) int64.  A negative token leaves its row out: its logits may hold anything, its
    outputs are 0 and so is its gradient.  A token from n on gives NaN.  (With `weight` a row that is left out takes
    as long as another.)
    temperature: a positive number, or a float32 tensor of one per row.

    A row of nothing but -inf gives -inf and the entropy 0; one with a NaN or +inf gives NaN.
    Where logits requires a gradient, logprobs and entropies carry it (token_logprobs_backward).  From
    hidden states there is no gradient: what requires one raises, unless under torch.no_grad()."""
    if weight is not None:
        return _made(TokenLogprobs, _ext().head_logprobs(x, weight, tokens, temperature, bool(entropy), _handle(stream)))
    if getattr(x, "requires_grad", False) and _torch().is_grad_enabled():
        out = _record(x, stream, "token_logprobs", tokens, temperature, (bool(entropy),), {"temperature": temperature})
        return TokenLogprobs(*out, temperature)
    return _made(TokenLogprobs, _ext().token_logprobs(x, tokens, temperature, bool(entropy), _handle(stream)))


def token_logprobs_backward(logits, tokens, r: TokenLogprobs, *, grad_logprobs=None, grad_entropies=None, out=None, stream=None):
    """Gradient of token_logprobs()'s logprobs and entropies with respect to the logits, in their type.

    grad_logprobs, grad_entropies: (rows,) float32, or None; the second needs a call with entropy=True.  A row
    whose entries are 0 gets 0, whatever its logits hold.  out: where to write, unit column stride; it may be the
    logits themselves.  Autograd takes it as changed in place: what has saved it raises when it is gone back
    through, and a leaf that requires a gradient is refused while gradients are recorded.  The result comes without a graph
    (an `out` as it is)."""
    if r.stats is None:
        raise ValueError("there is no gradient from hidden states: give logits")
    return _made(None, _ext().token_logprobs_backward(logits, tokens, r.temperature, r.stats, r.entropies, grad_logprobs, grad_entropies,
                                                      None, out, _handle(stream)))


def policy_loss(logits, tokens, old_logprobs, advantages, *, ref_logprobs=None, weights=None, temperature=1.0,
                clip_low: float = 0.2, clip_high: float = 0.2, kl: float = 0.0, entropy=None, gradient: bool = False, out=None,
                stream=None) -> PolicyLoss:
    """The clipped policy loss over tokens, with a KL term to a reference policy and an entropy bonus.

    With lp a token's log-probability (as token_logprobs gives it), r = exp(lp - old) and q = ref - lp:
        loss = sum of weights * (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl (exp(q) - 1 - q) - entropy H).
    logits, tokens, temperature: as in token_logprobs.  old_logprobs, advantages (A), ref_logprobs, weights:
    (rows,) float32, constants of the loss.  ref_logprobs None: no KL term.  weights: each token's factor, so
    mask / mask.sum() takes the mean over a mask and any other mean is as easy; 0 leaves a token out
    as a negative token does; None: 1 / rows.  entropy: its factor; None: entropies are not taken at all.

    Where logits requires a gradient, loss carries it (and going back reads the logits again: 4096 x 131072 bfloat16
    489 us in all, with gradient=True 339).  gradient=True gives grad_logits instead, the gradient
    of the loss in the logits' type, from the same launch (a second look at a row that is still on the chip); out: where
    to write it, as in token_logprobs_backward."""
    if not gradient and getattr(logits, "requires_grad", False) and _torch().is_grad_enabled():
        constants = {"old_logprobs": old_logprobs, "advantages": advantages, "ref_logprobs": ref_logprobs, "weights": weights,
                     "temperature": temperature}
        if out is not None:
            raise ValueError("out is for gradient=True")
        r = _record(logits, stream, "policy_loss", tokens, temperature,
                    (old_logprobs, advantages, ref_logprobs, weights, clip_low, clip_high, kl, entropy), constants)
        return PolicyLoss(*r, None, temperature)
    return _made(PolicyLoss, _ext().policy_loss(logits, tokens, old_logprobs, advantages, ref_logprobs, weights, temperature, clip_low,
                                                clip_high, kl, entropy, bool(gradient), out, _handle(stream)))


def policy_loss_backward(logits, tokens, r: PolicyLoss, *, grad_loss=None, out=None, stream=None):
    """Gradient of policy_loss()'s loss with respect to the logits, in their type.

    grad_loss: a float32 tensor of one element on the device; None: 1.  out: as in token_logprobs_backward."""
    return _made(None, _ext().token_logprobs_backward(logits, tokens, r.temperature, r.stats, r.entropies, r.slopes, r.entropy_slopes,
                                                      grad_loss, out, _handle(stream)))


def preference_loss(logits, tokens, offsets, *, ref_logprobs=None, beta: float = 0.1, label_smoothing: float = 0.0,
                    margin: float = 0.0, average: bool = False, temperature=1.0, stream=None) -> PreferenceLoss:
    """The preference loss of pairs of sequences, by their log-probabilities against a reference policy's.

    logits, tokens, temperature: as in token_logprobs; the rows of all sequences one behind the other, a negative
    token where a row does not count (a prompt's).  offsets: (2 pairs + 1,) int64 on the device, not falling:
    sequence j is the rows offsets[j] .. offsets[j + 1] - 1, 2i the one preferred to 2i + 1; rows before the first
    and behind the last are left out.  ref_logprobs: (rows,) float32, a constant, or None: 0.  With D_j
    the sum (average: the mean) of lp - ref over what counts of sequence j,
        d = beta (D_2i - D_2i+1) - margin,
    loss is the mean over the pairs of -(1 - e) log sigmoid(d) - e log sigmoid(-d), e the label_smoothing; margins
    holds the d.  Where an offset falls or leaves the rows, loss, all margins and the gradient of what is not left
    out are NaN.

    Where logits requires a gradient, loss carries it."""
    if getattr(logits, "requires_grad", False) and _torch().is_grad_enabled():
        r = _record(logits, stream, "preference_loss", tokens, temperature,
                    (offsets, ref_logprobs, beta, label_smoothing, margin, bool(average)),
                    {"ref_logprobs": ref_logprobs, "temperature": temperature})
        return PreferenceLoss(*r, temperature)
    return _made(PreferenceLoss, _ext().preference_loss(logits, tokens, offsets, ref_logprobs, beta, label_smoothing, margin, bool(average),
                                                        temperature, _handle(stream)))


def preference_loss_backward(logits, tokens, r: PreferenceLoss, *, grad_loss=None, out=None, stream=None):
    """Gradient of preference_loss()'s loss with respect to the logits, in their type.

    grad_loss: a float32 tensor of one element on the device; None: 1.  out: as in token_logprobs_backward."""
    return _made(None, _ext().token_logprobs_backward(logits, tokens, r.temperature, r.stats, None, r.slopes, None, grad_loss, out,
                                                      _handle(stream)))


def _record(logits, stream, name, tokens, temperature, args, constants):
    """The call under autograd: its outputs, of which the differentiable ones have a graph."""
    if stream is not None:
        raise ValueError("a call that records a gradient runs on the current stream: use torch.cuda.stream")
    for what, t in constants.items():
        if getattr(t, "requires_grad", False):
            raise ValueError(f"{what} counts as a constant, but requires a gradient: detach it")
    return _autograd().apply(logits, name, tokens, temperature, *args)


_function = None


def _autograd():
    """The autograd function behind the three calls, made on first use (torch is imported lazily)."""
    global _function
    if _function is None:
        torch = _torch()

        def gradient(logits, tokens, stats, entropies, slopes, entropy_slopes, temperature, scale):
            def plain(t):
                return None if t is None else t.detach().float().contiguous()
            return _made(None, _ext().token_logprobs_backward(logits.detach(), tokens, temperature, stats, entropies, plain(slopes),
                                                              plain(entropy_slopes), plain(scale), None, None))

        class Logprobs(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, name, tokens, temperature, *args):
                x = logits.detach()
                entropies = entropy_slopes = slopes = None
                if name == "token_logprobs":
                    out = _made(None, _ext().token_logprobs(x, tokens, temperature, *args, None))[:3]
                    _, entropies, stats = out
                    constants = (stats,)
                elif name == "policy_loss":
                    out = _made(None, _ext().policy_loss(x, tokens, *args[:4], temperature, *args[4:], False, None, None))[:9]
                    entropies, stats, slopes, entropy_slopes = out[5:]
                    constants = out[1:]
                else:
                    out = _made(None, _ext().preference_loss(x, tokens, *args, temperature, None))[:5]
                    _, margins, logprobs, stats, slopes = out
                    constants = (margins, logprobs, stats, slopes)
                ctx.mark_non_differentiable(*(t for t in constants if t is not None))
                ctx.set_materialize_grads(False)
                ctx.of_loss = name != "token_logprobs"
                per_row = isinstance(temperature, torch.Tensor)
                ctx.temperature = None if per_row else temperature
                ctx.inputs = 4 + len(args)
                ctx.save_for_backward(logits, tokens, stats, entropies, slopes, entropy_slopes, temperature if per_row else None)
                return out

            @staticmethod
            def backward(ctx, *grads):
                logits, tokens, stats, entropies, slopes, entropy_slopes, temperature = ctx.saved_tensors
                scale = None
                if ctx.of_loss:
                    scale = grads[0]
                    nothing = scale is None
                else:
                    slopes, entropy_slopes = grads[:2]
                    nothing = slopes is None and entropy_slopes is None
                if nothing:
                    return (None,) * ctx.inputs
                of = LogprobsGradient.apply if torch.is_grad_enabled() else gradient
                grad = of(logits, tokens, stats, entropies, slopes, entropy_slopes,
                          ctx.temperature if temperature is None else temperature, scale)
                return (grad,) + (None,) * (ctx.inputs - 1)

        class LogprobsGradient(torch.autograd.Function):
            """The gradient under create_graph: what is made of it leads back here, instead of counting as a constant."""

            @staticmethod
            def forward(ctx, *args):
                return gradient(*args)

            @staticmethod
            def backward(ctx, _grad):
                raise NotImplementedError("log-probabilities and the losses on them have no second derivative")
        _function = Logprobs
    return _function
