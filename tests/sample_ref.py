"""Truncated sampling in 64 bits, from its definition, on the CPU: per row, by sorting.

Tolerances. A whole-number mass is off by at most 2^-30 of itself (a table of 31 bits: 2^-32, a
polynomial of |q| < 2^-6.5 carried in 24 bits with five roundings: 5 * 2^-25 * 2^-6.5, its conversion
2^-32; the argument (x - max) / T * log2(e): products in pairs, 2^-24 * 2^-24 * 64, for bf16 logits
a difference that is exact or of a logit below 2^-12) or by one unit, 2^-43 of the largest for V up
to 2^20, whose mean is 0. A share of a sum is then off by less than 2^-29. SHARE is that: tokens and
numbers of tokens left are equal wherever no border is nearer."""
import math

import numpy as np
import torch

SHARE = 2.0 ** -29
# logp and log Z: a fp32 logarithm (its argument within one step of 2^-24, result within 1 ulp) and
# (x - max) / T with three roundings, then one of the difference
LOG_ABS = 2.0 ** -23
LOG_REL = 4 * 2.0 ** -24


def inv_T(T):
    return float(np.float32(1.0) / np.float32(T))


def row_truncation(x, T, k, p, mp):
    """x: 1-d float64 numpy of finite or -inf logits. Returns (order, kept, w in order, margin):
    `margin` is the least distance of a top-p border from p, as a share."""
    V = len(x)
    order = np.lexsort((np.arange(V), -x))
    xs = x[order]
    if T == 0 or p <= 0 or not math.isfinite(inv_T(T)):
        k, T, p = 1, 1.0, 1.0
    s = inv_T(T)
    w = np.exp((xs - xs[0]) * s)
    w[np.isneginf(xs)] = 0.0
    n = int((xs > -np.inf).sum())
    if k > 0:
        n = min(n, k)
    margin = math.inf
    if p < 1:
        c = np.concatenate([[0.0], np.cumsum(w[:n])])
        z = math.fsum(w[:n])
        n_p = max(1, int((c[:n] < p * z).sum()))
        margin = float(np.abs(c[1:n] / z - p).min()) if n > 1 else math.inf
        n = n_p
    if mp > 0:
        m = (xs[:n] - xs[0]) * s >= math.log(min(mp, 1.0))
        n = max(1, min(n, int(m.sum())))
    return order, n, w, margin


def row_draw(x, T, k, p, mp, u):
    """(token, logp, kept, mask, (m, log Z), margin of the truncation, margin of the draw)."""
    order, n, w, margin = row_truncation(x, T, k, p, mp)
    V = len(x)
    mass = np.zeros(V)
    mass[order[:n]] = w[:n]
    mask = np.zeros(V, bool)
    mask[order[:n]] = True
    z = math.fsum(w[:n])
    c = np.cumsum(mass)
    live = np.nonzero(mass > 0)[0]
    tok = int(live[np.searchsorted(c[live], u * c[-1], side="right").clip(max=len(live) - 1)])
    edges = np.abs(c[live][:-1] / c[-1] - u)
    s = inv_T(T) if T > 0 and math.isfinite(inv_T(T)) else 1.0
    at_max = float(x.max()) * s
    return (tok, (x[tok] - x.max()) * s - math.log(z), n, mask, (at_max, math.log(z)), margin,
            float(edges.min()) if len(edges) else math.inf)


def log_close(got, want):
    return abs(got - want) <= LOG_ABS + LOG_REL * abs(want)


def logits(rows, V, seed, dtype=torch.float32, std=2.0, peak=12.0):
    """Near-normal rows with some tokens that stand out, from flat to peaked."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, V, generator=g) * std
    n = min(V, 16)
    at = torch.randint(V, (rows, n), generator=g)
    h = torch.rand(rows, 1, generator=g) * peak
    x.scatter_add_(1, at, torch.rand(rows, n, generator=g) * h)
    return x.to(dtype)
