"""Infinite scores of tokens that a query sees: minus infinity is a weight of 0, plus
infinity is NaN, and a weight of 0 does not cancel a value that is not finite,
wherever in a tile the token lies.  Tolerances are those of test_gpu_paged_attn."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, host, to_dev
from oracle import attention as oa
from test_gpu_paged_attn import F16, I8, Setup, assert_close

pytestmark = pytest.mark.gpu


def put(s, at, k, v, seq=0):
    """Writes one token's key and value (all heads) of sequence `seq`."""
    rf.rfp2_kv_write(s.cache, to_dev(k[None].astype(np.float32)), to_dev(v[None].astype(np.float32)),
                     1, to_dev(np.array([seq], np.int32)), to_dev(np.array([at], np.int32)))


def without(s, at):
    """The reference with token `at` of sequence 0 left out."""
    s.k[0], s.v[0] = (np.delete(x, at, 0) for x in (s.k[0], s.v[0]))
    s.lens[0] -= 1
    return s.reference()


@pytest.mark.parametrize("D", [64, 96, 256])
@pytest.mark.parametrize("at", [5, 40, 149])
@pytest.mark.parametrize("small", [1.0, 2.0 ** -9, 2.0 ** -45])
def test_half_key_of_minus_infinity(D, at, small):
    """The query's value at the infinite key is an exact half, or far below the row's
    largest: its second half is 0, which must not be met by infinity."""
    announce("paged_attn -inf key", D, at, small)
    s = Setup(F16, [150, 33], 1, 4, 2, D, 16, seed=17)
    s.q = np.round(8 * s.q) / 8                               # every value an exact half
    s.q[0, 0, :, 3] = [small, -small, small, -small]
    k = s.k[0][at].copy()
    k[0, 3], k[1, 3] = -1e6, 1e6                              # held as -inf, +inf
    put(s, at, k, s.v[0][at])
    got = host(s.run())
    ref, tol = without(s, at)
    low = [0, 3]                  # heads 0, 1 read key head 0; heads 2, 3 read key head 1
    assert_close(got[0, 0, low], ref[0, 0, low], tol[0, 0, low])
    assert np.isnan(got[0, 0, [1, 2]]).all()                  # + infinity
    assert_close(got[1], ref[1], tol[1])


def test_half_key_of_infinity_against_zero_is_nan():
    announce("paged_attn inf key, zero query")
    s = Setup(F16, [150], 1, 2, 1, 64, 16, seed=18)
    s.q[0, 0, 1, 3] = 0.0
    s.q[0, 0, 0, 3] = 0.5
    k = s.k[0][70].copy()
    k[0, 3] = -1e6
    put(s, 70, k, s.v[0][70])
    got = host(s.run())
    assert np.isnan(got[0, 0, 1]).all() and np.isfinite(got[0, 0, 0]).all()


@pytest.mark.parametrize("fmt", [F16, I8])
@pytest.mark.parametrize("at", [40, 130, 149])
def test_zero_weight_does_not_cancel_a_value(fmt, at):
    """A token whose score is minus infinity, whose value is NaN: in the middle of a
    sequence, and in its last tile, where hidden values are taken out."""
    announce("paged_attn zero weight, NaN value", fmt, at)
    s = Setup(fmt, [150, 33], 1, 2, 1, 64, 16, seed=19)
    ref, tol = s.reference()
    s.q[0, 0, 0] = np.float32(2e30)                           # q.k beyond fp32
    s.q[0, 0, 1] = 0.001 * s.q[0, 0, 1]
    k, v = np.zeros((1, 64)), s.v[0][at].copy()
    n = s.lens[0]
    for t in range(n):                                        # keys that sum to 0 along the first query
        z = np.zeros((1, 64))
        z[0, :2] = [1.0, -1.0]
        s.k[0][t] = oa.held(z[None].astype(np.float32), fmt == I8)[0]
        put(s, t, z, s.v[0][t])
    k[0, :] = -1e10 if fmt == I8 else -6e4
    if fmt == F16:
        s.q[0, 0, 0] = np.float32(2e34)                       # 64 * 6e4 * 2e34 is beyond fp32
    v[0, 9] = np.nan
    put(s, at, k, v)
    got = host(s.run())
    lost = slice(0, 32) if fmt == I8 else slice(9, 10)
    assert np.isnan(got[0, 0, 0, lost]).all()
    rest = np.ones(64, bool)
    rest[lost] = False
    others = np.delete(s.v[0][:, 0], at, 0)[:, rest]           # equal weights: their mean
    err = np.abs(got[0, 0, 0, rest] - others.mean(0))
    assert np.all(err <= (np.sqrt(n) + 64) * 2.0 ** -24 * np.abs(others).mean(0)), err.max()
    assert_close(got[1], ref[1], tol[1])
