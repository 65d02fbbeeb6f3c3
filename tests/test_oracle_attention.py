"""Pins of the oracle's rotary positions, cache layout and attention."""
import math

import numpy as np
import pytest

from oracle import attention as oa


def test_rope_turns_by_the_angle_and_keeps_lengths():
    x = np.zeros((1, 1, 4), np.float32)
    x[0, 0] = [1.0, 0.0, 2.0, 5.0]
    f = np.array([0.5])
    y = oa.rope(x, [3], f, 2, interleaved=True)[0, 0]
    assert np.allclose(y, [math.cos(1.5), math.sin(1.5), 2.0, 5.0], atol=1e-15)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 16)).astype(np.float32)
    f = oa.rope_freqs(16, 10000.0)
    a, b = (oa.rope(x, np.arange(5), f, 16, i) for i in (False, True))
    assert np.array_equal(a[0], x[0]) and np.array_equal(b[0], x[0])     # position 0
    for y in (a, b):
        assert np.allclose((y ** 2).sum(-1), (x.astype(np.float64) ** 2).sum(-1))
    # the two styles are the same turn of differently paired values
    perm = np.stack([np.arange(8), np.arange(8) + 8], 1).reshape(-1)
    assert np.allclose(oa.rope(x[..., perm], np.arange(5), f, 16, True), a[..., perm])


def test_rope_scores_depend_on_distance_only():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 32)).astype(np.float32)
    f = oa.rope_freqs(32, 10000.0)
    dots = [float((oa.rope(q, [p + 7], f, 32, False) * oa.rope(k, [p], f, 32, False)).sum())
            for p in (0, 11, 100003)]
    assert np.allclose(dots, dots[0], atol=1e-9)


def test_rope_freqs_scaling():
    f = oa.rope_freqs(64, 10000.0)
    assert f[0] == 1.0 and np.all(np.diff(f) < 0)
    assert np.allclose(oa.rope_freqs(64, 10000.0, 8.0), f / 8)
    g = oa.rope_freqs(64, 10000.0, 8.0, 4096, 1.0, 32.0)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(g[turns >= 32], f[turns >= 32])
    assert np.allclose(g[turns <= 1], f[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(g[mid] < f[mid]) and np.all(g[mid] > f[mid] / 8)


def test_cache_layouts_place_every_token():
    x = np.arange(2 * 16 * 3 * 4).reshape(2, 16, 3, 4)
    k, v = oa.keys_in_memory(x), oa.eights_in_memory(x)
    for page, row, head, d in [(0, 0, 0, 0), (1, 7, 2, 3), (0, 8, 1, 2), (1, 15, 0, 1)]:
        assert k[page, head, row, d] == x[page, row, head, d]
        assert v.reshape(-1)[(((page * 3 + head) * 2 + row // 8) * 4 + d) * 8 + row % 8] \
            == x[page, row, head, d]


@pytest.mark.parametrize("window", [0, 1, 3])
def test_attention_by_hand_and_by_differences(window):
    """Against one score at a time; and d(y)/d(score) = w (v - y) by differences."""
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    y, _, _ = oa.attention(q, k, v, 6, 0.3, window)
    for h in range(4):
        js = [j for j in range(9) if j <= 6 and (not window or j > 6 - window)]
        w = [math.exp(0.3 * sum(q[h, i] * k[j, h // 2, i] for i in range(8))) for j in js]
        for i in range(8):
            assert math.isclose(y[h, i], sum(a * v[j, h // 2, i] for a, j in zip(w, js)) / sum(w),
                                rel_tol=1e-12, abs_tol=1e-13)
    e = 1e-6                        # moving key 5 along q raises its score by 0.3 |q|^2 e
    k2 = k.copy()
    k2[5, 0] += e * q[0]
    y2, _, _ = oa.attention(q, k2, v, 6, 0.3, window)
    w5 = (math.exp(0.3 * q[0] @ k[5, 0]) /
          sum(math.exp(0.3 * q[0] @ k[j, 0]) for j in range(9)
              if j <= 6 and (not window or j > 6 - window))) if window != 1 else 0.0
    assert np.allclose((y2[0] - y[0]) / e, 0.3 * (q[0] @ q[0]) * w5 * (v[5, 0] - y[0]), atol=1e-5)


def test_attention_sees_nothing_gives_zeros():
    q, k, v = np.ones((2, 8)), np.ones((0, 1, 8)), np.ones((0, 1, 8))
    assert not oa.attention(q, k, v, -1, 1.0)[0].any()
    assert not oa.attention(q, np.ones((3, 1, 8)), np.ones((3, 1, 8)), -1, 1.0)[0].any()


def test_turn_fractions_of_far_positions():
    assert abs(oa.turn_fraction(355, 1.0) - (355 / (2 * math.pi) - 57)) < 1e-13
    assert oa.turn_fraction(0, 0.3) == 0.0 and oa.turn_fraction(-5, 0.3) == -oa.turn_fraction(5, 0.3)
    # fractions add up modulo one, however far: p f = (p - 1) f + f
    for p in (1 << 20, (1 << 31) - 1, -(1 << 31)):
        for f in (1.0, 0.7498942093324559, 1e-4):
            d = oa.turn_fraction(p, f) - oa.turn_fraction(p - 1, f) - oa.turn_fraction(1, f)
            assert abs(d - round(d)) < 4e-16, (p, f, d)
    # and near the start both forms are the same rotation
    x = np.random.default_rng(3).standard_normal((4, 2, 16)).astype(np.float32)
    f = oa.rope_freqs(16, 10000.0)
    for i in (False, True):
        assert np.allclose(oa.rope(x, [0, 1, 2, 9], f, 16, i), oa.rope_far(x, [0, 1, 2, 9], f, 16, i),
                           rtol=0, atol=1e-14)
