"""The example's routed feed-forward part: norm, routing, expert products, gate and combine
together, against the oracle stage by stage, and as a replayed graph."""
import os
import sys

import numpy as np
import pytest

import bit_gemv_amd as rf
import oracle
from _gpu import announce, device, host, torch
from _layer import assert_codes, assert_rounded
from oracle import feed_forward as ff

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

WIDTH, INNER = 512, 256
ROUTERS = {
    "softmax": dict(top_k=4),
    "groups": dict(top_k=3, score=rf.ROUTE_SIGMOID, groups=4, group_top=2, top_groups=2, scale=2.5,
                   act=rf.GATE_GELU),
}


def make(tokens, kind, experts=16, seed=4):
    from moe_layer import MoeLayer
    g = torch.Generator(device=device())
    g.manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device=device())
    bias = 0.05 * normal(experts) if kind == "groups" else None
    layer = MoeLayer(0.1 * normal(experts, WIDTH), 0.06 * normal(experts, 2 * INNER, WIDTH),
                     0.06 * normal(experts, WIDTH, INNER), 1 + 0.1 * normal(WIDTH),
                     1 + 0.1 * normal(WIDTH), tokens, bias=bias, **ROUTERS[kind])
    layer.x.copy_(normal(tokens, WIDTH))
    layer.add.copy_(0.5 * normal(tokens, WIDTH))
    return layer


def within(y, packed, N, K, q, d, what):
    ref = oracle.ref_gemv(packed, N, K, q, d)
    assert np.all(np.abs(y - ref) <= 1e-5 * oracle.abs_product_sums(packed, N, K, q, d) + 1e-6), what


@pytest.mark.parametrize("kind", list(ROUTERS))
@pytest.mark.parametrize("tokens", [1, 2, 5, 40])
def test_step_against_the_oracle(tokens, kind):
    announce("moe layer", tokens, kind)
    layer = make(tokens, kind)
    E, k, T = layer.experts, layer.top_k, tokens
    kept = {}
    combine = rf.rfp2_moe_combine

    def watched(x, *args, **kw):             # the stream before it is added to in place
        kept["h"] = host(x).copy()
        combine(x, *args, **kw)
    rf.rfp2_moe_combine = watched
    try:
        layer.step()
    finally:
        rf.rfp2_moe_combine = combine
    # every stage from what the stage before gave, so that each is held to its own bound
    h = ff.add(host(layer.x), host(layer.add))
    assert np.array_equal(kept["h"], h)
    q, d = (host(t) for t in layer.acts_in)
    assert_codes(q, d, ff.rms_norm(h, host(layer.gain), layer.eps))
    logits = host(layer.logits)
    within(logits, host(layer.w_router).reshape(E, WIDTH // 32, 10), E, WIDTH, q, d, "router")
    ids, weights = host(layer.ids), host(layer.weights)
    bias, score, groups, group_top, top_groups, _, renorm, scale = layer.routing
    for t in range(T):
        want, w = ff.route(logits[t], None if bias is None else host(bias), score == rf.ROUTE_SIGMOID, groups,
                           group_top, top_groups, k, renorm, scale)
        assert ids[t].tolist() == want
        assert_rounded(weights[t], np.array(w))
    gate_up, down = host(layer.gate_up), host(layer.down)
    w_gu = host(layer.w_gate_up).reshape(E, 2 * INNER, WIDTH // 32, 10)
    w_down = host(layer.w_down).reshape(E, WIDTH, INNER // 32, 10)
    mid_q, mid_d = (host(t) for t in layer.acts_mid)
    assert_codes(mid_q, mid_d, ff.gated(gate_up[:, :INNER], gate_up[:, INNER:], layer.act == rf.GATE_GELU))
    for s, e in enumerate(ids.reshape(-1)):
        within(gate_up[s:s + 1], w_gu[e], 2 * INNER, WIDTH, q[s // k:s // k + 1], d[s // k:s // k + 1], "gate_up")
        within(down[s:s + 1], w_down[e], WIDTH, INNER, mid_q[s:s + 1], mid_d[s:s + 1], "down")
    rows = down.reshape(T, k, WIDTH)
    out = host(layer.h)
    assert_rounded(out, ff.combine(h, rows, weights),
                   np.abs(h) + (np.abs(weights)[..., None] * np.abs(rows)).sum(1))
    assert_codes(*(host(t) for t in layer.acts_out), ff.rms_norm(out, host(layer.next_gain), layer.eps))
    assert int(host(layer.err)[0]) == 0


@pytest.mark.parametrize("kind", list(ROUTERS))
@pytest.mark.parametrize("tokens", [1, 6, 33])
def test_replayed_graph_equals_eager_steps(tokens, kind):
    announce("moe layer graph", tokens, kind)
    eager, other = make(tokens, kind), make(tokens, kind)
    graph = other.capture()
    for layer in (eager, other):
        layer.x.copy_(make(tokens, kind, seed=5).x)
    for _ in range(5):
        eager.step()
        eager.x.copy_(eager.h)
        torch.cuda.synchronize()
        graph.replay()
        other.x.copy_(other.h)
        torch.cuda.synchronize()
        for a, b in zip((eager.h, eager.ids, eager.weights, *eager.acts_out),
                        (other.h, other.ids, other.weights, *other.acts_out)):
            assert torch.equal(a, b)


def test_two_graphs_and_a_padded_batch():
    """Two captured steps replayed on two streams at once, and a step whose last tokens are
    padding (logits of minus infinity): they get weights of 0 and keep their stream."""
    announce("moe layers at once")
    a, b = make(3, "softmax"), make(7, "groups")
    ga, gb = a.capture(), b.capture()
    a.step()
    b.step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (a.h, a.acts_out[0], b.h, b.acts_out[0])]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        for t in (a.h, a.acts_out[0], b.h, b.acts_out[0]):
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            ga.replay()
        with torch.cuda.stream(s2):
            gb.replay()
        torch.cuda.synchronize()
        for t, w in zip((a.h, a.acts_out[0], b.h, b.acts_out[0]), want):
            assert torch.equal(t, w)
    route = rf.rfp2_moe_route

    def padded(logits, *args, **kw):
        logits[1:] = -float("inf")
        route(logits, *args, **kw)
    rf.rfp2_moe_route = padded
    try:
        a.step()
    finally:
        rf.rfp2_moe_route = route
    assert int(host(a.err)[0]) == 0 and not host(a.weights)[1:].any()
    assert np.array_equal(host(a.h)[1:], ff.add(host(a.x), host(a.add))[1:])
    assert np.array_equal(host(a.h)[0], host(want[0])[0])
