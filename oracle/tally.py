"""Plain fp64 reference for the tally of attention weight and the eviction it decides.

TEST INFRASTRUCTURE ONLY -- never imported by the product package.

weight[t, g] is the sum, over the queries that attend token t and the query heads of KV
head g, of exp(s - lse).  An eviction keeps `budget` tokens of a head: the protected ones
(origin among the first `sinks` or the last `recent` of all the request's tokens), then the
largest weights, the lowest index first among equals; kept tokens of index >= budget move,
in order, into the free indices below it.
"""
from __future__ import annotations

import math

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def weights(q, k, lse, scale, positions):
    """q [n, Hq, D] at `positions` [n], k [L, H, D], lse [n, Hq] -> (w [L, H], err [L, H]):
    the weights, and sum of weight * sum_d |q_d k_d| * |scale| (what a rounding of a score
    is relative to).  NaN weights, those past fp32, and those of an lse of -inf or NaN, are
    nothing."""
    n, Hq, _ = q.shape
    L, H, _ = k.shape
    G = Hq // H
    w, err = np.zeros((L, H)), np.zeros((L, H))
    sees = np.arange(L)[:, None] <= np.asarray(positions)[None, :]  # [L, n]
    for h in range(Hq):
        g = h // G
        with np.errstate(all="ignore"):
            s = k[:, g] @ q[:, h].T * scale  # [L, n]
            size = np.abs(k[:, g]) @ np.abs(q[:, h]).T * abs(scale)
            p = np.exp(s - lse[:, h][None, :])
            p = np.where(sees & (p <= FLT_MAX) & (lse[:, h] > -math.inf)[None, :], p, 0.0)
        w[:, g] += p.sum(1)
        err[:, g] += np.where(p > 0, p * np.where(np.isfinite(size), size, 0), 0).sum(1)
    return w, err


def log_sum_exp(q, k, scale, positions):
    """lse [n, Hq] of queries at `positions` over keys 0 .. position."""
    n, Hq, _ = q.shape
    G = Hq // k.shape[1]
    out = np.full((n, Hq), -math.inf)
    for i in range(n):
        L = positions[i] + 1
        for h in range(Hq):
            s = k[:L, h // G] @ q[i, h] * scale
            if L > 0:
                m = s.max()
                out[i, h] = m + math.log(np.exp(s - m).sum())
    return out


def keep(weight, origin, total, budget, sinks, recent):
    """Indices of the kept tokens of one head, ascending (len(weight) > budget)."""
    def key(t):
        w = float(weight[t])
        if origin[t] < sinks or origin[t] >= total - recent:
            return (0, 0, 0.0, t)
        return (1, 1 if math.isnan(w) else 0, 0.0 if math.isnan(w) else -w, t)

    return sorted(sorted(range(len(weight)), key=key)[:budget])


def moves(kept, budget):
    """(from, to) pairs: the j-th kept token past the budget to the j-th free place."""
    inside = {t for t in kept if t < budget}
    free = [t for t in range(budget) if t not in inside]
    return list(zip([t for t in kept if t >= budget], free))
