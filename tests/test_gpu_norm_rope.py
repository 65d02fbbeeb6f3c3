"""Queries and keys normed head by head in the rows of a QKV product, then rotated and written
into the cache: the two calls in a row against the oracle, eagerly and as a replayed graph."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, host, to_dev, torch
from _layer import assert_rounded
from oracle import attention as oa
from oracle import feed_forward as ff

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.mark.parametrize("fmt", [rf.KV_F16, rf.KV_I8])
@pytest.mark.parametrize("T,H,KV,D", [(1, 8, 2, 128), (5, 4, 4, 64), (300, 6, 2, 96)])
def test_norm_then_rope_and_write(T, H, KV, D, fmt):
    announce("norm, rope, write", T, H, KV, D, fmt)
    rng = np.random.default_rng(T + D)
    rows = rng.standard_normal((T, (H + 2 * KV) * D)).astype(np.float32)
    gq, gk = ((1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2))
    pos, seq = np.arange(T, dtype=np.int32), np.zeros(T, dtype=np.int32)
    freqs = oa.rope_freqs(D, 10000.0)
    page = 16
    pages = -(-T // page)
    table = torch.arange(pages, dtype=torch.int32, device=device())[None]
    cache = rf.KvCache.allocate(fmt, pages, page, KV, D, table)
    source, g, sg, pg, fg = to_dev(rows), [to_dev(gq), to_dev(gk)], to_dev(seq), to_dev(pos), to_dev(freqs)
    qkv = source.clone()
    q, k, v = qkv.split([H * D, KV * D, KV * D], 1)
    out, kr, vr = (torch.empty(T, n, D, device=device()) for n in (H, KV, KV))

    def step():
        qkv.copy_(source)                    # a product's output
        rf.rfp2_rms_norm(q, T, H, D, g[0], EPS, q)
        rf.rfp2_rms_norm(k, T, KV, D, g[1], EPS, k)
        rf.rfp2_rope_kv_write(cache, q, k, v, T, H, sg, pg, fg, D, rf.ROPE_HALF, 1.0, out)
        rf.rfp2_kv_read(cache, T, sg, pg, kr, vr)
    step()
    x = rows.reshape(T, H + 2 * KV, D)
    normed = host(qkv).reshape(T, H + 2 * KV, D)
    assert_rounded(normed[:, :H], ff.rms_norm(x[:, :H], gq, EPS))
    assert_rounded(normed[:, H:H + KV], ff.rms_norm(x[:, H:H + KV], gk, EPS))
    assert np.array_equal(normed[:, H + KV:], x[:, H + KV:])           # the values are left alone
    turned = oa.rope(normed[:, :H + KV], pos, freqs, D, False).astype(np.float32)
    assert np.array_equal(host(out), turned[:, :H])
    # code times scale, once rounded
    assert_rounded(host(kr), oa.held(turned[:, H:], fmt == rf.KV_I8))
    assert_rounded(host(vr), oa.held(x[:, H + KV:], fmt == rf.KV_I8))
    want = [t.clone() for t in (out, kr, vr)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(3):
        for t in (out, kr, vr, cache.k, cache.v):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, kr, vr), want))
