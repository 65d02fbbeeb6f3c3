"""Rotation and cache calls over more tokens than one launch holds (2^32 threads at
most): a workgroup of 256 threads a token, or for eight.  Most tokens are zeros or
padding; those around the borders of launches and at the end are looked at."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, host, to_dev, torch
from oracle import attention as oa

pytestmark = pytest.mark.gpu


def looked_at(T, borders):
    """Token numbers: the start, around every border, the end."""
    at = [np.arange(9), np.arange(T - 9, T)] + [b + np.arange(-5, 5) for b in borders if b < T - 20]
    return np.unique(np.concatenate(at))


def test_rope():
    T = (1 << 24) + 5
    announce("rope of many tokens", T)
    at = looked_at(T, [1 << 20, 3 << 20, 1 << 23])
    rng = np.random.default_rng(0)
    part = rng.standard_normal((len(at), 1, 4)).astype(np.float32)
    x = torch.zeros(T, 1, 4, device=device())
    rows = to_dev(at)
    x[rows] = to_dev(part)
    pos = torch.arange(T, dtype=torch.int32, device=device())
    f = oa.rope_freqs(4, 10000.0)
    y = torch.full_like(x, -5.0)
    rf.rfp2_rope(x, T, 1, 4, pos, to_dev(f), 4, rf.ROPE_HALF, 1.0, y)
    ref = oa.rope_far(part, at, f, 4, False)
    assert np.all(np.abs(host(y[rows]) - ref) <= 2.0 ** -24 * np.abs(ref) + 2.0 ** -48 * 8)
    y[rows] = 0
    assert not bool(y.any())


@pytest.mark.parametrize("fmt", [rf.KV_F16, rf.KV_I8])
def test_cache(fmt):
    T, D, P, launch = (1 << 27) + 4099, 32, 16, 8 * ((1 << 20) - 2)
    announce("kv_write/read of many tokens", fmt, T)
    at = looked_at(T, [launch, 2 * launch, 1 << 26, 16 * launch])
    rng = np.random.default_rng(1)
    part = rng.standard_normal((len(at), 1, D)).astype(np.float32)
    x = torch.zeros(T, 1, D, device=device())                 # keys and values alike
    rows = to_dev(at)
    x[rows] = to_dev(part)
    pages = -(-len(at) // P)
    c = rf.KvCache.allocate(fmt, pages, P, 1, D, to_dev(rng.permutation(pages).astype(np.int32)[None]))
    seq = torch.zeros(T, dtype=torch.int32, device=device())
    pos = torch.full((T,), -1, dtype=torch.int32, device=device())
    pos[rows] = torch.arange(len(at), dtype=torch.int32, device=device())
    err = torch.zeros(1, dtype=torch.int32, device=device())
    rf.rfp2_kv_write(c, x, x, T, seq, pos, err)
    k = torch.full_like(x, -5.0)
    rf.rfp2_kv_read(c, T, seq, pos, k, x, err)
    held = oa.held(part, fmt == rf.KV_I8).astype(np.float32)
    for got in (k, x):
        assert np.array_equal(host(got[rows]), held)
        got[rows] = 0
        assert not bool(got.any())                            # padding reads as zeros
    assert int(host(err)[0]) == 0
    del c, x, k, got, seq, pos
    torch.cuda.empty_cache()
