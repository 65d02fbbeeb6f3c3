"""A place of the cache that several tokens of one call name: a mixture of theirs,
element by element, and nothing else is touched."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, host, to_dev, torch
from test_gpu_kv_cache import expected, make_cache, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [rf.KV_F16, rf.KV_I8])
@pytest.mark.parametrize("T", [90, 2500])
def test_a_place_named_several_times(fmt, T):
    announce("kv_write, places named several times", fmt, T)
    H, D, P = 3, 64, 16
    rng = np.random.default_rng(T)
    x = np.exp2(rng.integers(-6, 6, (2, T, 1, 1))) * rng.standard_normal((2, T, H, D))
    k, v = x.astype(np.float32)
    pos = np.arange(T, dtype=np.int32)
    for a, b in ((3, 40), (3, T - 1), (17, 18), (64, 71)):    # b names a's place, its own stays empty
        pos[b] = pos[a]
    pages = -(-T // P) + 1
    table = rng.permutation(pages)[None].astype(np.int32)
    c = make_cache(fmt, pages, P, H, D, table)
    err = torch.zeros(1, dtype=torch.int32, device=device())
    rf.rfp2_kv_write(c, to_dev(k), to_dev(v), T, to_dev(np.zeros(T, np.int32)), to_dev(pos), err)
    assert int(host(err)[0]) == 0
    got = [host(t) for t in (c.k, c.v)] + ([host(t) for t in (c.k_scale, c.v_scale)] if fmt == rf.KV_I8 else [])
    # the memory had every named place been written by its first, second, .. last token
    twice = sorted({int(p) for p in pos if (pos == p).sum() > 1})
    turns = []
    for i in range(3):
        keep = np.ones(T, bool)
        for p in twice:
            names = np.flatnonzero(pos == p)
            keep[names] = False
            keep[names[min(i, len(names) - 1)]] = True
        turns.append(expected(fmt, pages, P, H, D, table, k[keep], v[keep],
                              np.zeros(keep.sum(), np.int32), pos[keep]))
    for g, refs in zip(got, zip(*turns)):
        bits = lambda a: np.ascontiguousarray(a).view({1: np.uint8, 2: np.uint16, 4: np.uint32}[a.itemsize])
        assert np.all((bits(g) == bits(refs[0])) | (bits(g) == bits(refs[1])) | (bits(g) == bits(refs[2])))
        same = (bits(refs[0]) == bits(refs[1])) & (bits(refs[0]) == bits(refs[2]))
        assert same_bits(g[same], refs[0][same])
