"""The example's decode layer: products, rotation, cache and attention together,
against the oracle step by step, and as a replayed graph."""
import os
import sys

import numpy as np
import pytest

import bit_gemv_amd as rf
import oracle
from _gpu import announce, device, host, torch
from oracle import attention as oa

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

HEADS, KV, D, WIDTH, SEQS = 8, 2, 64, 512, 3


def make(fmt, lens):
    from decode_layer import DecodeLayer
    g = torch.Generator(device=device())
    g.manual_seed(3)

    def normal(*s):
        return torch.randn(*s, generator=g, device=device())
    layer = DecodeLayer(0.05 * normal((HEADS + 2 * KV) * D, WIDTH), 0.05 * normal(WIDTH, HEADS * D),
                        HEADS, KV, D, SEQS, 80, fmt, page_size=16)
    k, v = normal(SEQS, 70, KV, D), normal(SEQS, 70, KV, D)
    layer.fill(k, v, lens)
    layer.x.copy_(normal(SEQS, WIDTH))
    return layer, host(k), host(v)


@pytest.mark.parametrize("fmt", [rf.KV_F16, rf.KV_I8])
def test_step_against_the_oracle(fmt):
    announce("decode layer", fmt)
    lens, i8 = [70, 0, 33], fmt == rf.KV_I8
    layer, k, v = make(fmt, lens)
    freqs = oa.rope_freqs(D, 10000.0)
    held = [[oa.held(x[s, :n], i8) if n else np.zeros((0, KV, D)) for x in (k, v)]
            for s, n in enumerate(lens)]
    for _ in range(3):
        layer.step()
        # every stage from what the stage before gave, so that each is held to its own bound
        qkv, q, attn, out = (host(t) for t in (layer.qkv, layer.q, layer.attn, layer.out))
        for x, w, N, K, y in ((host(layer.x), layer.w_qkv, layer.rows, WIDTH, qkv),
                              (attn, layer.w_out, WIDTH, HEADS * D, out)):
            qa, da = oracle.quantize_acts(x)
            packed = host(w).reshape(N, K // 32, 10)
            ref = oracle.ref_gemv(packed, N, K, qa, da)
            assert np.all(np.abs(y - ref) <= 1e-5 * oracle.abs_product_sums(packed, N, K, qa, da) + 1e-6)
        rows = qkv.reshape(SEQS, HEADS + 2 * KV, D)
        turned = oa.rope(rows[:, :HEADS + KV], lens, freqs, D, False)
        assert np.array_equal(q.reshape(SEQS, HEADS, D), turned[:, :HEADS].astype(np.float32))
        for s in range(SEQS):
            new = turned[s, HEADS:].astype(np.float32), rows[s, HEADS + KV:]
            held[s] = [np.concatenate([h, oa.held(n[None], i8)]) for h, n in zip(held[s], new)]
            ref, mag, big = oa.attention(q[s].reshape(HEADS, D), *held[s], lens[s], D ** -0.5)
            tol = mag * ((2 * big * (4 * D ** 0.5 + 16) + 80) * 2.0 ** -24)[:, None]
            assert np.all(np.abs(attn[s].reshape(HEADS, D) - ref) <= tol)
        lens = [n + 1 for n in lens]
        layer.x.copy_(layer.out)
    assert host(layer.lens).tolist() == lens and int(host(layer.err)[0]) == 0


@pytest.mark.parametrize("fmt", [rf.KV_F16, rf.KV_I8])
def test_replayed_graph_equals_eager_steps(fmt):
    announce("decode layer graph", fmt)
    eager, _, _ = make(fmt, [60, 5, 0])
    other, _, _ = make(fmt, [60, 5, 0])
    graph = other.capture()
    for _ in range(6):
        eager.step()
        eager.x.copy_(eager.out)
        torch.cuda.synchronize()
        graph.replay()
        other.x.copy_(other.out)
        torch.cuda.synchronize()
        assert torch.equal(eager.out, other.out) and torch.equal(eager.lens, other.lens)
