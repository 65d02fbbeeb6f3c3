"""Rotary positions far out, against angles reduced in whole numbers.

The angle's fraction of a turn is off by a few units of 2^-53 at any position, which
is 2 pi times that in radians, and the cosine, the sine and the two products add as
much again: 2^-48 of the pair's size holds all of it.  The value is then rounded once
(2^-24 of it)."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, empty, host, to_dev, torch
from oracle import attention as oa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [4000, 123457, 1 << 20, (1 << 27) - 31, (1 << 31) - 64, -(1 << 31)])
@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (38, False)])
def test_far_positions_keep_their_angle(first, rot, inter):
    announce("rope far", first, rot, inter)
    T, H, D = 64, 3, 128
    rng = np.random.default_rng(rot)
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    pos = (first + np.arange(T)).astype(np.int32)
    f = oa.rope_freqs(rot, 10000.0)
    ref = oa.rope_far(x, pos, f, rot, inter, 1.25)
    ref[..., rot:] = x[..., rot:]
    y = empty((T, H, D), torch.float32)
    rf.rfp2_rope(to_dev(x), T, H, D, to_dev(pos), to_dev(f), rot,
                 rf.ROPE_INTERLEAVED if inter else rf.ROPE_HALF, 1.25, y)
    err = np.abs(host(y).astype(np.float64) - ref)
    tol = 2.0 ** -24 * np.abs(ref) + 2.0 ** -48 * 1.25 * 2 * np.abs(x).max()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), err[bad].max(), np.argwhere(bad)[:4])
