"""Routing among scores far below one: cases, and the definition in decimals of 60 digits,
whose exponents do not end where fp64's do (not collected by pytest)."""
from __future__ import annotations

from decimal import Decimal, getcontext

import numpy as np

getcontext().prec = 60
INF = float("inf")


def weights(logits, ids, sigmoid, scale):
    """scale * p / (sum of the chosen p) of the chosen experts; 0 where all are masked."""
    def score(x):                              # up to a softmax's common factor
        if x == -INF:
            return Decimal(0)
        e = Decimal(float(x) - top).exp()
        return e / (1 + Decimal(float(x)).exp()) if sigmoid else e
    chosen = [float(logits[i]) for i in ids]
    top = max([x for x in chosen if x != -INF], default=0.0)
    p = [score(x) for x in chosen]
    total = sum(p)
    return [float(Decimal(scale) * x / total) if total else 0.0 for x in p]


def cases():
    """name, logits, bias or None, sigmoid, groups, group_top, top_groups, top_k, scale, ids."""
    far = np.full(8, -900.0, dtype=np.float32)
    far[[1, 4, 6]] = -700.0, -702.5, -701.25
    yield "sigmoids of -700", far, None, True, 1, 1, 1, 3, 1.0, [1, 6, 4]
    edge = np.full(70, -800.0, dtype=np.float32)
    edge[[3, 69, 20]] = -689.5, -690.25, -691.0
    yield "sigmoids around -690", edge, None, True, 1, 1, 1, 3, 2.5, [3, 69, 20]
    beyond = np.full(300, -2000.0, dtype=np.float32)
    beyond[[299, 0, 150]] = -1000.0, -1001.0, -1000.5
    yield "sigmoids beyond fp64", beyond, None, True, 1, 1, 1, 4, 1.0, [299, 150, 0, 1]
    yield "sigmoids of the lowest number", np.full(64, np.finfo(np.float32).min), None, True, 1, 1, 1, 6, 1.0, [
        0, 1, 2, 3, 4, 5]
    bias = np.full(70, -1.0, dtype=np.float32)
    bias[[3, 20, 69]] = 0.3, 0.1, 0.2
    yield "sigmoids around -690 with a bias", edge, bias, True, 1, 1, 1, 3, 1.0, [3, 69, 20]
    # a softmax's largest is what the bias keeps away
    one = np.zeros(128, dtype=np.float32)
    one[5] = 800.0
    one[[7, 100]] = 1.5, -0.75
    away = np.zeros(128, dtype=np.float32)
    away[[5, 7, 100, 64]] = -9.0, 0.3, 0.25, 0.125
    yield "softmax without its largest", one, away, False, 1, 1, 1, 3, 1.0, [7, 100, 64]
    one = one.copy()
    one[5] = 30000.0
    # groups of 32 count 0.3 + 0, 0 + 0, 0.125 + 0 and 0.25 + 0: the first and the last stay, and
    # of their experts without a bias the lowest comes third
    yield "softmax far below its largest", one, away, False, 4, 2, 2, 3, 1.0, [7, 100, 0]
    masked = np.full(16, -INF, dtype=np.float32)
    masked[[2, 9]] = -750.0, -751.0
    yield "two of -750 and masks", masked, None, True, 1, 1, 1, 4, 1.0, [2, 9, 0, 1]
    yield "only masks", np.full(16, -INF, dtype=np.float32), None, True, 1, 1, 1, 4, 1.0, [0, 1, 2, 3]
    for low in (-340.0, -346.0, -347.0, -350.0):       # where fp64's scores give way to the logits
        step = np.arange(32, dtype=np.float32) * -0.625 + np.float32(low)
        yield f"sigmoids from {low} down", step, None, True, 1, 1, 1, 32, 1.0, list(range(32))
