"""The selections of a language model by their definitions, in float64 numpy.

``token``, ``routing`` and ``routed`` restate the formulas one row or one batch at a time,
by full sorts and plain sums; ``routing_gradient`` is the derivative written out
per token from the Jacobians.  Used by tests only.
"""
from __future__ import annotations

import numpy as np


def order_of(values):
    """Indices in the library order: descending, ties by lower index, without -inf and NaN."""
    v = np.asarray(values)
    live = np.flatnonzero(v > -np.inf)
    return live[np.argsort(-v[live] + 0.0, kind="stable")]


def scaled(l, m, T):
    """(l - m) / T, 0 where l == m (an infinite maximum included)."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        d = np.where(l == m, 0.0, l - m)
        return np.where(d == 0, 0.0, np.where(d == -np.inf, -np.inf, d / T))


def _kept(l, allowed, T, k, p, min_p):
    """The kept tokens in the library order, their x and w (p and min_p: numbers)."""
    order = order_of(np.where(allowed, l, -np.inf))
    if not order.size:
        return order, order, order
    if 0 < k < order.size:
        order = order[:k]
    x = scaled(l[order], l[order[0]], T)
    w = np.exp(x)
    keep = x > -np.inf
    if p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        keep &= before < p * w.sum()
        keep[0] = True
    keep &= w >= min(min_p, 1.0)
    return order[keep], x[keep], w[keep]


def _scores(x, q):
    with np.errstate(invalid="ignore", divide="ignore"):
        score = x - np.log(np.asarray(q, np.float64))
    return np.where(np.isnan(score), -np.inf, score)


def _refused(l, allowed, T, p, min_p):
    return not T >= 0 or np.isnan(p) or np.isnan(min_p) or np.isnan(l[allowed]).any()


def token(logits, noise, allowed, T, k, p, min_p):
    """(token, logprob) of one row."""
    l = np.asarray(logits, np.float64)
    if _refused(l, allowed, T, p, min_p):
        return -1, np.nan
    order, x, w = _kept(l, allowed, T if T > 0 else 1.0, k if T > 0 else 1, p, min_p)
    if not order.size:
        return -1, -np.inf
    score = _scores(x, noise[order])
    winner = order[score == score.max()].min()
    return int(winner), float(x[order == winner][0] - np.log(w.sum()))


def tokens_within(logits, noise, allowed, T, k, p, min_p, score_blur, mass_blur):
    """{token: (lowest logprob, highest)}: what one row may give when scores are
    within score_blur of their values, and masses and weights within mass_blur
    (relative).  One entry where the decision is clear."""
    l = np.asarray(logits, np.float64)
    if T == 0 or _refused(l, allowed, T, p, min_p):
        t, lp = token(logits, noise, allowed, T, k, p, min_p)
        return {t: (lp, lp)}
    order, x, w = _kept(l, allowed, T, k, p + mass_blur if p < 1 else p, min_p * (1 - mass_blur) if min_p < 1 else 1.0)
    if not order.size:
        return {-1: (-np.inf, -np.inf)}
    inner = _kept(l, allowed, T, k, p - mass_blur if p < 1 else p, min_p * (1 + mass_blur) if min_p < 1 else 1.0)[0].size
    score = _scores(x, noise[order])
    least = score[:inner].max()
    if np.isinf(least):
        may = order == order[:inner][score[:inner] == least].min()
    else:
        may = score >= least - score_blur
        for v in np.unique(x[may]):  # of equal logits with equal noise, the lowest index in any precision
            same = np.flatnonzero(may & (x == v))
            for q in np.unique(score[same]):
                equal = same[score[same] == q]
                may[equal[order[equal] != order[equal].min()]] = False
    hi, lo = -np.log(w[:inner].sum()), -np.log(w.sum())
    return {int(t): (v + lo, v + hi) for t, v in zip(order[may], x[may])}


def _log_scores(z, score):
    if score == "sigmoid":
        return np.minimum(z, 0.0) - np.log1p(np.exp(-np.abs(z)))
    return z


def _softmax(y):
    """Along the last axis; copies of an infinite maximum share the mass."""
    e = np.exp(scaled(y, y.max(-1, keepdims=True), 1.0))
    return e / e.sum(-1, keepdims=True)


def routing(z32, k, score, normalize, bias=None, mask=None):
    """gates, experts, counts, loss of float32 logits z32 (tokens, experts)."""
    z32 = np.asarray(z32, np.float32)
    with np.errstate(invalid="ignore"):
        c = z32 if bias is None else z32 + np.asarray(bias, np.float32)  # a float32 sum, by definition
    experts = np.full((len(z32), k), -1, np.int64)
    for t in range(len(z32)):
        if mask is None or mask[t]:
            chosen = order_of(c[t])[:k]
            experts[t, :chosen.size] = chosen
    gates, counts, loss = routed(z32, experts, score, normalize)
    return gates, experts, counts, loss


def scores_and_bias(z32, score, bias):
    """What the choice is by where the bias is added to the scores, in float64 (-inf where the logit is)."""
    z = np.asarray(z32, np.float32).astype(np.float64)
    y = _log_scores(z, score)
    s = np.exp(y) if score == "sigmoid" else np.stack([_softmax(row) if row.max() > -np.inf else 0 * np.exp(row) for row in y])
    return np.where(z == -np.inf, -np.inf, s + np.asarray(bias, np.float64))


def routed(z32, experts, score, normalize):
    """gates, counts, loss of float32 logits z32 (tokens, experts) for a choice (-1: an empty slot, the last ones)."""
    z = np.asarray(z32, np.float32).astype(np.float64)
    E = z.shape[1]
    gates = np.zeros(experts.shape)
    P = np.zeros(E)
    for t in range(len(z)):
        chosen = experts[t][experts[t] >= 0]
        if not chosen.size:
            continue
        y = _log_scores(z[t], score)
        p = np.full(E, np.nan) if np.isnan(z[t]).any() else _softmax(y)
        g = _softmax(y[chosen]) if normalize else p[chosen] if score == "softmax" else np.exp(y[chosen])
        gates[t, :chosen.size] = np.nan if np.isnan(z[t]).any() else g
        P += chosen.size * p
    counts = np.bincount(experts[experts >= 0], minlength=E)
    N = max(int(counts.sum()), 1)
    return gates, counts, float(E * ((counts / N) * (P / N)).sum())


def routing_gradient(z32, experts, counts, score, normalize, grad_gates=None, grad_loss=None):
    """d(sum grad_gates * gates + grad_loss * loss) / dz, choice and counts constant."""
    z = np.asarray(z32, np.float32).astype(np.float64)
    tokens, E = z.shape
    N = max(int(counts.sum()), 1)
    out = np.zeros_like(z)
    for t in range(tokens):
        chosen = experts[t][(experts[t] >= 0) & (experts[t] < E)]
        if not chosen.size:
            continue
        y = _log_scores(z[t], score)
        p = _softmax(y)
        J = np.diag(p) - np.outer(p, p)  # dp / dy
        dy = np.zeros(E)
        if grad_loss is not None:
            dy += J @ (grad_loss * E * (counts / N) * chosen.size / N)
        if grad_gates is not None:
            dg = grad_gates[t][(experts[t] >= 0) & (experts[t] < E)]
            if normalize:
                g = _softmax(y[chosen])
                dy[chosen] += (np.diag(g) - np.outer(g, g)) @ dg
            elif score == "softmax":
                dy += J[:, chosen] @ dg
            else:
                dy[chosen] += np.exp(y[chosen]) * dg
        if score == "sigmoid":
            dy *= np.exp(-np.maximum(z[t], 0) - np.log1p(np.exp(-np.abs(z[t]))))  # sigmoid(-z)
        out[t] = dy
    return out
