"""Tolerances of the log-probability kernels, and inputs for them.

A row's exponents x = (l - m) / T carry two roundings of float32 (2^-23 |x|), the hardware's 2^x two units
(2^-22), and a sum of them the additions of a chunk, of a warp and of the CTAs (at most 32, 2^-19): so
  s  is off by at most 2^-18 + 2^-23 (mean |x|) of itself, the mean by the probabilities, and with it
  log s by as much and its rounding,
  a log-probability by that and 2^-22 |x| + 2^-24 |value|,
  an entropy by that and 2^-18 of mean |x|.
A gradient g (1 - p) - h p (...) is off by what p is, times the size of its terms, and by its rounding to the
logits' type (half a step, and half the smallest subnormal step of float16).  A 2^x below 2^-126 counts as zero, and
its factor is that of p with a sum of at least 1: where the terms' size over T is above 1, the loss is 2^-126 times it.
"""
import numpy as np
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def sizes(l, T):
    """Each row's largest finite |x| of anything likely, and its mean by the probabilities."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        z = l / np.broadcast_to(np.asarray(T, np.float64), len(l))[:, None]
        x = z - np.max(z, 1, keepdims=True, initial=-np.inf)
        e = np.exp(x)
        e = np.where(np.isnan(e), 0.0, e)
        mean = np.where(e > 0, -x * e, 0.0).sum(1) / np.maximum(e.sum(1), 1e-300)
    return np.where(np.isfinite(x), -x, 0.0), mean


def row_error(mean, x=0.0, value=0.0):
    return 2.0 ** -18 + 2.0 ** -22 * (mean + np.abs(x)) + 2.0 ** -23 * np.abs(value)


def gradient_error(l, T, g, h, want, dtype):
    x, mean = sizes(l, T)
    T = np.broadcast_to(np.asarray(T, np.float64), len(l))[:, None]
    p = np.exp(-x)
    p = np.where(np.isfinite(l), p, 0.0)
    p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    g, h = np.abs(g)[:, None], np.abs(0.0 if h is None else h)
    h = h[:, None] if np.ndim(h) else h
    off = row_error(mean)[:, None] + 2.0 ** -22 * x
    terms = g + h * (x + mean[:, None] + np.log(l.shape[1]))
    return p * terms / T * 2 * off + 2.0 ** -126 * terms / T + 2.0 ** -22 * np.abs(want) + HALF_STEP[dtype] * np.abs(want) * 1.01 + TINY[dtype] + 2.0 ** -24 * (g * (p > 0.5)) / T


def close(got, want, off, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bad = ~((np.abs(got - want) <= off) | (got == want) | (np.isnan(got) & np.isnan(want)))
    if bad.any():
        i = np.unravel_index(np.flatnonzero(bad)[0], bad.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; first at {i}: {got[i]} instead of {want[i]}, "
                             f"allowed {np.broadcast_to(off, got.shape)[i]}")


def as_numpy(t):
    return t.detach().double().cpu().numpy()


def make(rows, n, dtype, ld=0, seed=0, left_out=0.0, device="cuda", spread=3.0, offset=0):
    """Logits of rows of n (stride ld, beginning `offset` elements behind a boundary) and a token for each row."""
    g = torch.Generator(device=device).manual_seed(1000 * seed + n)
    ld = ld or n
    store = torch.randn(rows * ld + offset + 16, generator=g, device=device).mul_(spread).to(dtype)
    logits = store[offset:offset + rows * ld].view(rows, ld)[:, :n]
    tokens = torch.randint(n, (rows,), generator=g, device=device)
    if left_out:
        tokens = torch.where(torch.rand(rows, generator=g, device=device) < left_out, -1, tokens)
    return logits, tokens, g
