"""What the tests of the norm, gate and combine calls share (not collected by pytest)."""
from __future__ import annotations

import numpy as np

STEP = 2.0 ** -24        # half a step of fp32, relative to the value


def assert_rounded(y, ref, size=0.0, what=""):
    """fp64 arithmetic rounded once to fp32: half a step of the value, plus the inner
    roundings (up to 2^10 of them at 2^-53 of `size`, the sum of the terms' magnitudes) and
    half a step of the smallest numbers."""
    y, ref = np.asarray(y, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    err = np.abs(y - ref)
    bad = ~(err <= STEP * np.abs(ref) + 2.0 ** -43 * (np.abs(ref) + size) + 2.0 ** -150)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:5].tolist(), err[bad][:5], ref[bad][:5])


def assert_codes(q, d, ref, what=""):
    """int8 codes and scales of fp32(ref): d = fl(max / 127) of a rounded max (two
    half steps, and half a step of the smallest numbers twice); a code is the rounding of
    fl(fl(ref) / d) (two half steps of a ratio of up to 127.5)."""
    M, K = ref.shape
    b = np.asarray(ref, dtype=np.float64).reshape(M, K // 32, 32)
    amax = np.abs(b).max(-1)
    d = np.asarray(d, dtype=np.float64).reshape(M, K // 32)
    bad = ~(np.abs(d - amax / 127) <= 2.01 * STEP * amax / 127 + 2.0 ** -149)
    assert not bad.any(), (what, "scales", int(bad.sum()), np.argwhere(bad)[:5].tolist())
    q = np.asarray(q, dtype=np.float64).reshape(b.shape)
    assert np.abs(q).max() <= 127
    far = np.abs(q * d[..., None] - b) > (0.5 + 127.5 * 2.01 * STEP) * d[..., None] + 2.0 ** -149
    far &= (d > 2.0 ** -126)[..., None]                  # below, a step of d itself is the larger error
    assert not far.any(), (what, "codes", int(far.sum()), np.argwhere(far)[:5].tolist())
