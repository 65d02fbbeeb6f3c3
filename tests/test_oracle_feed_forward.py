"""Pins of the oracle's norms, routing, gate activation and weighted sum (CPU only)."""
import math
from fractions import Fraction

import numpy as np

from oracle import feed_forward as ff


def test_rms_norm_by_hand_and_by_invariants():
    # mean of squares of (3, 4) is 12.5
    assert np.allclose(ff.rms_norm([[3.0, 4.0]], [1.0, 2.0], 0.0),
                       [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]], rtol=1e-15)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 96))
    y = ff.rms_norm(x, np.ones(96), 0.0)
    assert np.allclose((y * y).mean(-1), 1.0, rtol=1e-14)
    assert np.allclose(ff.rms_norm(7.0 * x, np.ones(96), 0.0), y, rtol=1e-14)
    # eps alone: a row of zeros stays zeros, a tiny one is divided by sqrt(eps)
    assert not ff.rms_norm(np.zeros((1, 8)), np.ones(8), 1e-6).any()
    assert np.allclose(ff.rms_norm(np.full((1, 8), 1e-20), np.ones(8), 1e-6), 1e-17, rtol=1e-12)


def test_add_rounds_once():
    x, a = np.float32(1.0), np.float32(2.0 ** -25)
    assert ff.add([x], [a])[0] == 1.0 and ff.add([x], [np.float32(3 * 2.0 ** -25)])[0] == np.float32(1 + 2.0 ** -23)


def test_combine_against_fractions():
    rng = np.random.default_rng(1)
    x, r = rng.standard_normal((2, 4)).astype(np.float32), rng.standard_normal((2, 3, 4)).astype(np.float32)
    w = rng.standard_normal((2, 3)).astype(np.float32)
    h = ff.combine(x, r, w)
    for t in range(2):
        for k in range(4):
            want = Fraction(float(x[t, k])) + sum(Fraction(float(w[t, j])) * Fraction(float(r[t, j, k])) for j in range(3))
            assert abs(h[t, k] - float(want)) <= 8 * 2.0 ** -53 * (
                abs(float(x[t, k])) + sum(abs(float(w[t, j]) * float(r[t, j, k])) for j in range(3)))
    assert np.array_equal(ff.combine(None, r, w) + 0.0, ff.combine(np.zeros((2, 4)), r, w))


def test_gate_activations():
    g = np.array([0.0, 1.0, -1.0, 40.0, -800.0])
    silu = ff.gated(g, np.ones(5), False)
    assert silu[0] == 0 and abs(silu[1] - 1 / (1 + math.exp(-1))) < 1e-15 and silu[3] == 40.0 and silu[4] == 0
    assert abs(silu[1] + silu[2] - (silu[1] - 1 / (1 + math.e))) < 1e-15           # silu(-1) = -1 / (1 + e)
    gelu = ff.gated(g, np.full(5, 2.0), True)
    # printed to six places in many tables: gelu(1) = 0.841192 in the tanh form
    assert abs(gelu[1] / 2 - 0.841192) < 5e-7 and abs(gelu[2] / 2 + 0.158808) < 5e-7 and gelu[3] == 80.0
    # the definition by tanh where its sum does not cancel, and its tail exp(2 z) where it does
    for x in (0.7, 3.0, -0.4):
        z = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
        assert abs(float(ff.gated([x], [1.0], True)[0]) - 0.5 * x * (1 + math.tanh(z))) < 1e-15
    z = math.sqrt(2 / math.pi) * (-9 - 0.044715 * 729)
    assert abs(float(ff.gated([-9.0], [1.0], True)[0]) / (-9 * math.exp(2 * z)) - 1) < 1e-12


def test_scores():
    assert np.allclose(ff.scores([0.0, math.log(3.0)], False), [0.25, 0.75], rtol=1e-15)
    assert ff.scores([-math.inf, 5.0], False) == [0.0, 1.0]
    assert ff.scores([-math.inf, -math.inf], False) == [0.0, 0.0]
    assert np.allclose(ff.scores([0.0, math.log(3.0), -math.inf, -1e30], True), [0.5, 0.75, 0.0, 0.0])
    assert ff.scores([0.0, -690.0, -690.5], False)[2] == 0.0 < ff.scores([0.0, -690.0, -690.5], False)[1]


def test_route_by_hand():
    l = [1.0, 3.0, 3.0, 0.0]
    ids, w = ff.route(l, None, False, 1, 1, 1, 3, True, 2.0)
    assert ids == [1, 2, 0]                                    # the lower first among equals
    e = math.exp(-2.0)
    assert np.allclose(w, [2 / (2 + e), 2 / (2 + e), 2 * e / (2 + e)], rtol=1e-15)
    # a bias changes the choice, not the weights
    ids, w = ff.route([0.0, 0.0, 0.0], [0.0, 0.1, 0.2], True, 1, 1, 1, 2, False, 1.0)
    assert ids == [2, 1] and w == [0.5, 0.5]
    # groups of two by their largest and by their sum: (4, 0) against (3, 3)
    l = [math.log(x) for x in (4.0, 1e-9, 3.0, 3.0)]
    assert ff.route(l, None, False, 2, 1, 1, 1, True, 1.0)[0] == [0]
    assert ff.route(l, [0.0] * 4, False, 2, 2, 1, 1, True, 1.0)[0] == [2]
    # masked experts come last, with weight 0
    ids, w = ff.route([-math.inf, 2.0, -math.inf, -math.inf], None, False, 1, 1, 1, 3, True, 1.0)
    assert ids == [1, 0, 2] and w == [1.0, 0.0, 0.0]
    ids, w = ff.route([-math.inf] * 3, None, True, 1, 1, 1, 2, True, 1.0)
    assert ids == [0, 1] and w == [0.0, 0.0]
    # a group counts by what of it is not masked
    l = [-math.inf, 2.0, 0.1, 0.2]
    assert ff.route(l, [0.0] * 4, True, 2, 2, 1, 2, True, 1.0)[0] == [3, 2]
    assert ff.route([-math.inf, 2.0, -math.inf, 1.0], [0.0] * 4, True, 2, 2, 1, 1, True, 1.0)[0] == [1]
