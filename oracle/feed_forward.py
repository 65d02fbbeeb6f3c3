"""Plain fp64 statement of the calls around the products of a feed-forward part:
norms, routing, the gate's activation and the experts' weighted sum.

What a call rounds to fp32 before it goes on (the residual stream, the values that are
quantized) is rounded here too; everything else is fp64, one value or one expert at a time
where that is the plainer way to say it.
"""
from __future__ import annotations

import math

import numpy as np


def rms_norm(x, gain, eps):
    """x [..., K] -> fp64 (not rounded)."""
    x = np.asarray(x, dtype=np.float64)
    mean = np.array([math.fsum(r * r) / r.size for r in x.reshape(-1, x.shape[-1])])
    inv = 1.0 / np.sqrt(mean + eps)
    return x * inv.reshape(x.shape[:-1] + (1,)) * np.asarray(gain, dtype=np.float64)


def add(x, a):
    """The residual stream after a product's rows were added to it, fp32."""
    return (np.asarray(x, dtype=np.float64) + np.asarray(a, dtype=np.float64)).astype(np.float32)


def combine(x, rows, weights):
    """x [T][K] or None, rows [T][k][K], weights [T][k] -> fp64 (not rounded)."""
    h = np.zeros(rows[:, 0].shape) if x is None else np.asarray(x, dtype=np.float64)
    for j in range(rows.shape[1]):
        h = h + np.asarray(weights[:, j, None], dtype=np.float64) * np.asarray(rows[:, j], dtype=np.float64)
    return h


def gated(g, u, gelu):
    """act(g) * u, fp64 (not rounded)."""
    g, u = np.asarray(g, dtype=np.float64), np.asarray(u, dtype=np.float64)
    # 0.5 (1 + tanh z) is written as 1 / (1 + exp(-2 z)): the same number, but for z < 0 the
    # sum 1 + tanh z cancels (at z = -18 nothing is left of it in 53 bits)
    z = 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3) if gelu else g
    with np.errstate(over="ignore", invalid="ignore"):     # an infinite gate gives NaN
        return g / (1.0 + np.exp(-z)) * u


def scores(logits, sigmoid):
    """One token's scores; a logit of minus infinity scores 0, and so does one whose
    exponential is below exp(-690)."""
    l = [float(x) for x in logits]
    if sigmoid:
        return [0.0 if x < -690.0 else 1.0 / (1.0 + math.exp(-x)) for x in l]
    top = max(l)
    e = [0.0 if x == -math.inf or x - top < -690.0 else math.exp(x - top) for x in l]
    total = math.fsum(e)
    return [x / total if total else 0.0 for x in e]


def shares(logits, p):
    """The chosen experts' scores p over their sum; 0 where all are masked.  Of scores so small
    that fp64 loses some, the exponentials over the largest one's: there a sigmoid's 1 / (1 + e^l)
    is 1 within 2^-499, and a softmax's sum is the same for all."""
    total = math.fsum(p)
    if total < 2.0 ** -500:
        top = max(logits)
        p = [0.0 if l == -math.inf else math.exp(float(l) - float(top)) for l in logits]
        total = math.fsum(p)
    return [x / total if total else 0.0 for x in p]


def route(logits, bias, sigmoid, groups, group_top, top_groups, top_k, renorm, scale):
    """One token -> (ids, fp64 weights)."""
    E = len(logits)
    p = scores(logits, sigmoid)
    v = [-math.inf if x == -math.inf else float(x) if bias is None else p[e] + float(bias[e])
         for e, x in enumerate(logits)]
    per = E // groups
    value = []
    for g in range(groups):
        best = sorted((x for x in v[g * per:(g + 1) * per] if x != -math.inf), reverse=True)
        value.append(math.fsum(best[:group_top]) if best else -math.inf)
    kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
    there = [e for e in range(E) if e // per in kept]
    ids = sorted(there, key=lambda e: (-v[e], e))[:top_k]
    w = [p[e] for e in ids]
    if renorm:
        w = shares([logits[e] for e in ids], w)
    return ids, [scale * x for x in w]
