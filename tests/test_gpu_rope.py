"""GPU parity of the rotary positions: frequencies and rotation against the fp64 oracle.

The rotation is computed in fp64 and rounded once: half a step of fp32, 2^-24
of the value, plus what the angle's own fp64 rounding moves (positions to 2^20
times a few units of 2^-53 a turn: below 2^-30 of the pair's size)."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, empty, host, to_dev, torch
from oracle import attention as oa

pytestmark = pytest.mark.gpu


def assert_rounded(y, ref, x, mscale):
    size = abs(mscale) * np.abs(x.astype(np.float64)).max() * 2
    err = np.abs(y.astype(np.float64) - ref)
    bad = ~(err <= 2.0 ** -24 * np.abs(ref) + 2.0 ** -30 * size)
    assert not bad.any(), (bad.sum(), err[bad][:5], np.argwhere(bad)[:5])


@pytest.mark.parametrize("args", [(2, 10000.0, 1.0, 0.0, 0.0, 1.0), (128, 500000.0, 1.0, 0.0, 0.0, 1.0),
                                  (96, 10000.0, 4.0, 0.0, 0.0, 1.0),
                                  (1024, 10000.0, 16.0, 4096.0, 1.0, 32.0),
                                  (6, 100.0, 2.5, 17.0, 0.0, 0.5)])
def test_freqs(args):
    announce("rope_freqs", args)
    f = empty(args[0] // 2 + 1, torch.float64)
    f.fill_(-7.0)
    rf.rfp2_rope_freqs(*args, f)
    got, ref = host(f), oa.rope_freqs(*args)
    assert got[-1] == -7.0                                   # nothing past the end
    # pow is within a few units of 2^-53 of its result, and the parts' sums likewise
    assert np.all(np.abs(got[:-1] - ref) <= 2.0 ** -48 * ref)


CASES = [  # T, H, D, rot, interleaved, first position, factor
    (1, 1, 4, 2, False, 0, 1.0), (1, 40, 128, 128, False, 1000, 1.0), (7, 3, 128, 64, True, 65535, 8.0),
    (33, 8, 64, 64, True, 5, 1.0), (5, 2, 96, 22, False, 131071, 1.0), (5, 2, 96, 22, True, 131071, 4.0),
    (3, 17, 256, 256, False, 1 << 20, 1.0), (2, 1, 1024, 1024, True, 1 << 20, 1.0),
    (2, 5, 20, 6, False, -9, 1.0), (300, 6, 128, 120, False, 0, 1.0), (1, 64, 192, 190, True, 12, 1.0),
    (600, 3, 128, 128, False, 9, 1.0), (530, 5, 64, 32, True, 70000, 4.0), (512, 2, 96, 30, False, 3, 1.0),
]


@pytest.mark.parametrize("T,H,D,rot,inter,first,factor", CASES)
def test_rope(T, H, D, rot, inter, first, factor):
    announce("rope", T, H, D, rot, inter, first, factor)
    rng = np.random.default_rng(T * 1000 + D)
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    pos = (first + rng.permutation(T)).astype(np.int32)
    f = oa.rope_freqs(rot, 10000.0, factor, 4096.0, 1.0, 32.0)
    m = 1.0 if factor == 1.0 else 1.25
    ref = oa.rope(x, pos, f, rot, inter, m)
    ref[..., rot:] = x[..., rot:]
    xg, pg, fg = to_dev(x), to_dev(pos), to_dev(f)
    style = rf.ROPE_INTERLEAVED if inter else rf.ROPE_HALF
    y = empty((T, H, D), torch.float32)
    rf.rfp2_rope(xg, T, H, D, pg, fg, rot, style, m, y)
    got = host(y)
    assert_rounded(got, ref, x, m)
    assert np.array_equal(got[..., rot:], x[..., rot:])
    assert np.array_equal(host(xg), x)                       # inputs are never written
    # rows that lie apart, on a stream of its own, and in place
    wide = torch.full((T, H * D + 8), -3.0, device=device())
    out = torch.full((T, H * D + 4), -5.0, device=device())
    wide[:, :H * D] = xg.reshape(T, H * D)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    rf.rfp2_rope(wide, T, H, D, pg, fg, rot, style, m, out, s)
    rf.rfp2_rope(wide, T, H, D, pg, fg, rot, style, m, wide, s)
    w, o = host(wide), host(out)
    assert np.array_equal(o[:, :H * D].reshape(T, H, D), got)
    assert np.array_equal(w[:, :H * D].reshape(T, H, D), got)
    assert (w[:, H * D:] == -3.0).all() and (o[:, H * D:] == -5.0).all()


def test_rope_passes_infinities_and_nan_to_their_pair_only():
    announce("rope non-finite")
    x = np.ones((1, 1, 64), np.float32)
    x[0, 0, 3], x[0, 0, 40] = np.inf, np.nan
    f = to_dev(oa.rope_freqs(64, 10000.0))
    y = empty((1, 1, 64), torch.float32)
    rf.rfp2_rope(to_dev(x), 1, 1, 64, to_dev(np.array([5], np.int32)), f, 64, rf.ROPE_HALF, 1.0, y)
    bad = np.flatnonzero(~np.isfinite(host(y)[0, 0]))
    assert set(bad) == {3, 35, 8, 40}
