"""The norm, combine, routing and gate calls beyond what one launch holds and beyond 32-bit
offsets: rows at both ends and around the borders against small calls on the same rows
(which other tests hold to the oracle)."""
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, torch

pytestmark = pytest.mark.gpu
EPS = 1e-5
MANY = (1 << 20) + 5                        # rows of a launch, and a few


def normal(*shape, seed=1):
    g = torch.Generator(device())
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=device())


def some(T):
    """Rows at the ends and around the border of a launch."""
    return sorted({r for r in (0, 1, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, T // 2, T - 1) if 0 <= r < T})


def test_many_rows_of_the_norms():
    announce("norms, many rows")
    K, T, at = 32, MANY, some(MANY)
    x, a, gain = normal(T, K), normal(T, K, seed=2), normal(K, seed=3)
    h, y = torch.empty_like(x), torch.empty_like(x)
    q, d = torch.empty(T, K, dtype=torch.int8, device=device()), torch.empty(T, 1, device=device())
    rf.rfp2_add_rms_norm(x, a, T, K, gain, EPS, h, y, q, d)
    n = len(at)
    h2, y2 = torch.empty(n, K, device=device()), torch.empty(n, K, device=device())
    q2, d2 = torch.empty(n, K, dtype=torch.int8, device=device()), torch.empty(n, 1, device=device())
    rf.rfp2_add_rms_norm(x[at], a[at], n, K, gain, EPS, h2, y2, q2, d2)
    for big, small in ((h, h2), (y, y2), (q, q2), (d, d2)):
        assert torch.equal(big[at], small)
    rows, w = normal(T, 2, K, seed=4), normal(T, 2, seed=5)
    rf.rfp2_moe_combine(x, rows, w, T, 2, K, h, gain, EPS, y, q, d)
    rf.rfp2_moe_combine(x[at], rows[at], w[at], n, 2, K, h2, gain, EPS, y2, q2, d2)
    for big, small in ((h, h2), (y, y2), (q, q2), (d, d2)):
        assert torch.equal(big[at], small)
    alone = torch.empty_like(h)
    rf.rfp2_moe_combine(x, rows, w, T, 2, K, alone)
    assert torch.equal(alone, h)
    rf.rfp2_rms_norm(x, T, 2, 16, gain[:16].clone(), EPS, y)
    rf.rfp2_rms_norm(x[at], n, 2, 16, gain[:16].clone(), EPS, y2)
    assert torch.equal(y[at], y2)


def test_many_heads():
    announce("norm of many heads")
    H = 4 * ((1 << 20) + 3)                  # more workgroups of heads than a launch holds along y
    x, gain = normal(1, H * 4), normal(4, seed=2)
    y = torch.empty_like(x)
    rf.rfp2_rms_norm(x[:, :1 << 24], 1, 1 << 22, 4, gain, EPS, y[:, :1 << 24])
    for h in (0, 1, 32 * 65535 - 1, 32 * 65535, 32 * 65535 + 1, (1 << 22) - 1):
        one = torch.empty(1, 4, device=device())
        rf.rfp2_rms_norm(x[:, 4 * h:4 * h + 4].clone(), 1, 1, 4, gain, EPS, one)
        assert torch.equal(y[:, 4 * h:4 * h + 4], one), h


@pytest.mark.parametrize("E,groups", [(2, 1), (8, 2)])
def test_many_tokens_routed(E, groups):
    announce("routing of many tokens", E, groups)
    T, at = MANY, some(MANY)
    l, bias = normal(T, E), normal(E, seed=2)
    args = (bias, rf.ROUTE_SIGMOID, groups, 1, 1, 2, True, 1.5)
    ids, w = torch.empty(T, 2, dtype=torch.int32, device=device()), torch.empty(T, 2, device=device())
    rf.rfp2_moe_route(l, T, E, *args, ids, w)
    i2, w2 = torch.empty(len(at), 2, dtype=torch.int32, device=device()), torch.empty(len(at), 2, device=device())
    rf.rfp2_moe_route(l[at], len(at), E, *args, i2, w2)
    assert torch.equal(ids[at], i2) and torch.equal(w[at], w2)
    assert int(ids.min()) >= 0 and int(ids.max()) < E


def test_offsets_beyond_32_bits():
    """Rows that lie 2^31 values and more from the first: far apart, and many of them."""
    announce("offsets beyond 32 bits")
    K, far = 96, (1 << 30) + 64
    wide = torch.zeros(3 * far, device=device())
    x = wide.as_strided((3, K), (far, 1))
    x.copy_(normal(3, K))
    gain, near = normal(K, seed=2), x.clone()
    y, y2 = torch.empty(3, K, device=device()), torch.empty(3, K, device=device())
    q, q2 = (torch.empty(3, K, dtype=torch.int8, device=device()) for _ in range(2))
    d, d2 = (torch.empty(3, K // 32, device=device()) for _ in range(2))
    rf.rfp2_add_rms_norm(x, x, 3, K, gain, EPS, None, y, q, d)
    rf.rfp2_add_rms_norm(near, near, 3, K, gain, EPS, None, y2, q2, d2)
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(d, d2)
    rf.rfp2_rms_norm(x, 3, 3, 32, gain[:32].clone(), EPS, y)
    rf.rfp2_rms_norm(near, 3, 3, 32, gain[:32].clone(), EPS, y2)
    assert torch.equal(y, y2)
    rf.rfp2_quantize_gated_acts(x, x, 3, K, rf.GATE_SILU, q, d)
    rf.rfp2_quantize_gated_acts(near, near, 3, K, rf.GATE_SILU, q2, d2)
    assert torch.equal(q, q2) and torch.equal(d, d2)
    i, i2 = (torch.empty(3, 4, dtype=torch.int32, device=device()) for _ in range(2))
    w, w2 = torch.empty(3, 4, device=device()), torch.empty(3, 4, device=device())
    rf.rfp2_moe_route(x, 3, K, None, rf.ROUTE_SOFTMAX, 1, 1, 1, 4, True, 1.0, i, w)
    rf.rfp2_moe_route(near, 3, K, None, rf.ROUTE_SOFTMAX, 1, 1, 1, 4, True, 1.0, i2, w2)
    assert torch.equal(i, i2) and torch.equal(w, w2)


def test_more_than_2_to_31_values():
    announce("2^31 values and more")
    k, K = 8, 4096
    T = (1 << 31) // (k * K) + 3
    rows = torch.empty(T, k, K, device=device())
    for t in range(0, T, 4096):
        rows[t:t + 4096].normal_()
    w, h = normal(T, k), torch.empty(T, K, device=device())
    rf.rfp2_moe_combine(None, rows, w, T, k, K, h)
    at = [0, T // 2, T - 4, T - 3, T - 2, T - 1]
    h2 = torch.empty(len(at), K, device=device())
    rf.rfp2_moe_combine(None, rows[at], w[at], len(at), k, K, h2)
    assert torch.equal(h[at], h2)
    del h
    # the same memory as gate and up rows: 2^31 values of each half and the codes of them
    M, W = T * k // 2, K
    gate = rows.view(-1)[:2 * M * W].view(M, 2 * W)
    q, d = torch.empty(M, W, dtype=torch.int8, device=device()), torch.empty(M, W // 32, device=device())
    rf.rfp2_quantize_gated_acts(gate[:, :W], gate[:, W:], M, W, rf.GATE_GELU, q, d)
    at = [0, M // 2, M - 2, M - 1]
    q2, d2 = torch.empty(4, W, dtype=torch.int8, device=device()), torch.empty(4, W // 32, device=device())
    rf.rfp2_quantize_gated_acts(gate[at][:, :W], gate[at][:, W:], 4, W, rf.GATE_GELU, q2, d2)
    assert torch.equal(q[at], q2) and torch.equal(d[at], d2)


def test_more_codes_than_a_launch_holds():
    announce("2^32 codes read back")
    K = 4096
    M = (1 << 32) // K + 3
    q = torch.zeros(M, K, dtype=torch.int8, device=device())
    d = torch.zeros(M, K // 32, device=device())
    at = [0, 1, M // 2, M - 4, M - 3, M - 1]
    q[at] = (torch.arange(K, device=device()) % 255 - 127).to(torch.int8)
    d[at] = normal(len(at), K // 32)
    a = torch.empty(M, K, device=device())
    rf.rfp2_dequantize_acts(q, d, M, K, a)
    want = q[at].float().view(len(at), K // 32, 32) * d[at][..., None]
    assert torch.equal(a[at], want.view(len(at), K))
    assert not a[2].any() and not a[M - 2].any()


@pytest.mark.parametrize("K", [1024, 2048, 4096, 5120, 8192, 16384, 20000, 70016])
@pytest.mark.parametrize("values", [1 << 20, 1 << 24])
def test_rows_past_the_caches(K, values):
    """Each width class with outputs, and with rows too, that go past the caches, in place:
    the bits of small calls."""
    announce("norms past the caches", K, values)
    T = values // K + 2
    x, a, gain = normal(T, K), normal(T, K, seed=2), normal(K, seed=3)
    quant = K % 32 == 0
    at = [0, 1, T // 2, T - 1]
    h2, y2 = (torch.empty(4, K, device=device()) for _ in range(2))
    codes = ((torch.empty(T, K, dtype=torch.int8, device=device()), torch.empty(T, K // 32, device=device()))
             if quant else (None, None))
    few = ((torch.empty(4, K, dtype=torch.int8, device=device()), torch.empty(4, K // 32, device=device()))
           if quant else (None, None))
    xs, as_ = x[at], a[at]
    rf.rfp2_add_rms_norm(xs, as_, 4, K, gain, EPS, h2, y2, *few)
    rf.rfp2_add_rms_norm(x, a, T, K, gain, EPS, x, a, *codes)           # h over x, y over add
    assert torch.equal(x[at], h2) and torch.equal(a[at], y2)
    assert not quant or all(torch.equal(b[at], s) for b, s in zip(codes, few))
    rf.rfp2_add_rms_norm(h2, None, 4, K, gain, EPS, None, y2)
    rf.rfp2_add_rms_norm(x, None, T, K, gain, EPS, None, x)
    assert torch.equal(x[at], y2)
    w, rows, y = normal(T, 1, seed=6), normal(T, K, seed=7), torch.empty_like(x)
    rf.rfp2_moe_combine(y2, rows[at], w[at], 4, 1, K, h2, gain, EPS, xs)
    rf.rfp2_moe_combine(x, rows, w, T, 1, K, x, gain, EPS, y)           # onto the stream in place
    assert torch.equal(x[at], h2) and torch.equal(y[at], xs)


def rounded(y, ref):
    """Half a step of fp32 and of its smallest numbers, and the fp64 arithmetic."""
    return bool(((y.double() - ref).abs() <= (2.0 ** -24 + 2.0 ** -43) * ref.abs() + 2.0 ** -150).all())


def test_the_widest_rows():
    announce("rows of 2^24 values")
    K = 1 << 24
    x, a, gain = normal(1, K), normal(1, K, seed=2), normal(K, seed=3)
    h, y = torch.empty_like(x), torch.empty_like(x)
    q, d = torch.empty(1, K, dtype=torch.int8, device=device()), torch.empty(1, K // 32, device=device())
    rf.rfp2_add_rms_norm(x, a, 1, K, gain, EPS, h, y, q, d)
    assert torch.equal(h, x + a)
    t = h.double()
    assert rounded(y, t / torch.sqrt((t * t).mean() + EPS) * gain.double())
    q2, d2 = torch.empty_like(q), torch.empty_like(d)
    rf.rfp2_quantize_acts(y, 1, K, q2, d2)
    assert torch.equal(q, q2) and torch.equal(d, d2)
    rf.rfp2_moe_combine(x, a, torch.ones(1, 1, device=device()), 1, 1, K, h, gain, EPS, None, q2, d2)
    assert torch.equal(h, x + a) and torch.equal(q, q2) and torch.equal(d, d2)
    rf.rfp2_quantize_gated_acts(x, a, 1, K, rf.GATE_SILU, q, d)
    g = x.double()
    rf.rfp2_quantize_acts((g / (1 + torch.exp(-g)) * a.double()).float(), 1, K, q2, d2)
    assert torch.equal(d, d2) and torch.equal(q, q2)
    rf.rfp2_dequantize_acts(q, d, 1, K, y)
    assert torch.equal(y, (q.view(-1, 32).float() * d.view(-1, 1)).view(1, K))


@pytest.mark.parametrize("T,k,K", [(1, 1024, 64), (3, 1024, 4096), (1000, 1, 32)])
def test_the_most_rows_a_token(T, k, K):
    announce("combine of many rows", T, k, K)
    x, rows, w, h = normal(T, K), normal(T, k, K, seed=2), normal(T, k, seed=3), torch.empty(T, K, device=device())
    rf.rfp2_moe_combine(x, rows, w, T, k, K, h)
    terms = w.double()[..., None] * rows.double()
    ref = x.double() + terms.sum(1)
    size = x.double().abs() + terms.abs().sum(1)
    # one rounding to fp32; k + 1 terms in fp64, in any order, on either side
    assert bool(((h.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 2 * (k + 2) * 2.0 ** -53 * size).all())
