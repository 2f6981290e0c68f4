"""Log-probabilities of given tokens and the losses on them, from their definitions in float64.

Test infrastructure: shares no code with the library.  Rows are numpy arrays; a row whose token is negative
(or that a loss leaves out) has the values 0 and the gradient 0.
"""
from __future__ import annotations

import numpy as np


def row(l, token, T):
    """(logprob, entropy, p, logp) of one row."""
    z = np.asarray(l, np.float64) / T
    m = z.max()
    if m == -np.inf:
        return -np.inf, 0.0, np.zeros_like(z), np.full_like(z, -np.inf)
    if not m < np.inf:
        return np.nan, np.nan, np.full_like(z, np.nan), np.full_like(z, np.nan)
    logp = z - m - np.log(np.exp(z - m).sum())
    p = np.exp(logp)
    H = -(p[p > 0] * logp[p > 0]).sum()
    return (logp[token] if token < len(z) else np.nan), H, p, logp


def logprobs(l, tokens, T=1.0):
    """(logprobs, entropies) of all rows; T a number or one per row."""
    T = np.broadcast_to(np.asarray(T, np.float64), len(tokens))
    got = [row(l[r], t, T[r])[:2] if t >= 0 else (0.0, 0.0) for r, t in enumerate(tokens)]
    return tuple(np.array(v, np.float64) for v in zip(*got)) if got else (np.zeros(0), np.zeros(0))


def gradient(l, tokens, T, g, h=None):
    """Of sum g logprob + h entropy by the logits; rows whose g and h are 0 get 0."""
    T = np.broadcast_to(np.asarray(T, np.float64), len(tokens))
    h = np.zeros(len(tokens)) if h is None else h
    out = np.zeros(l.shape, np.float64)
    for r, t in enumerate(tokens):
        if t < 0 or (g[r] == 0 and h[r] == 0):
            continue
        _, H, p, logp = row(l[r], t, T[r])
        if not p.any():
            continue
        d = -g[r] * p - h[r] * p * np.where(p > 0, logp + H, 0.0)
        if t < len(p):
            d[t] += g[r]
        else:
            d[:] = np.nan
        out[r] = d / T[r]
    return out


def policy(lp, H, old, A, ref, w, live, low, high, kl, entropy):
    """(loss, kl sum, clipped weight, entropy sum, d loss / d logprob, d loss / d entropy)."""
    ratio = np.exp(lp - old)
    inside = np.clip(ratio, 1 - low, 1 + high) * A
    clipped = inside < ratio * A
    term, slope = -np.minimum(ratio * A, inside), np.where(clipped, 0.0, -A * ratio)
    k3 = np.zeros_like(lp)
    if ref is not None:
        q = ref - lp
        k3 = np.exp(q) - 1 - q
        term, slope = term + kl * k3, slope - kl * (np.exp(q) - 1)
    term = term - entropy * H
    w = np.where(live, w, 0.0)
    take = lambda v: np.where(live, w * v, 0.0)  # noqa: E731
    return take(term).sum(), take(k3).sum(), w[clipped & live].sum(), take(H).sum(), take(slope), take(np.full_like(lp, -entropy))


def preference(lp, tokens, offsets, ref, beta, smoothing=0.0, margin=0.0, average=False):
    """(loss, margins, d loss / d logprob): lp is 0 where a row does not count."""
    pairs, live = len(offsets) // 2, np.asarray(tokens) >= 0
    ratio = np.where(live, lp - (0.0 if ref is None else ref), 0.0)
    D, share = [], []
    for a, b in zip(offsets[:-1], offsets[1:]):
        share.append(1.0 / max(1, live[a:b].sum()) if average else 1.0)
        D.append(share[-1] * ratio[a:b].sum())
    D = np.array(D)
    d = beta * (D[0::2] - D[1::2]) - margin
    soft = lambda v: np.logaddexp(0.0, v)  # noqa: E731
    terms = (1 - smoothing) * soft(-d) + smoothing * soft(d)
    each = beta / max(pairs, 1) * (smoothing / (1 + np.exp(-d)) - (1 - smoothing) / (1 + np.exp(d)))
    slope = np.zeros(len(lp))
    for j, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
        slope[a:b] = np.where(live[a:b], (-each[j // 2] if j % 2 else each[j // 2]) * share[j], 0.0)
    return (terms.mean() if pairs else 0.0), d, slope
