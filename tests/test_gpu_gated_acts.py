"""GPU parity of the quantized gate activation and of the values that int8 activations
stand for, against the fp64 oracle."""
import numpy as np
import pytest

import bit_gemv_amd as rf
import oracle
from _gpu import announce, device, empty, host, to_dev, torch
from _layer import assert_codes
from oracle import feed_forward as ff

pytestmark = pytest.mark.gpu

SIZES = [(1, 32), (8, 1536), (3, 96), (33, 2048), (7, 4128), (1, 14336), (1100, 64), (600, 1536), (2, 65536),
         (5, 160)]


def run(g, u, act, M, K):
    q = torch.full((M + 1, K), 99, dtype=torch.int8, device=device())
    d = torch.full((M + 1, K // 32), -7.0, device=device())
    rf.rfp2_quantize_gated_acts(g, u, M, K, act, q, d)
    assert (host(q)[M] == 99).all() and (host(d)[M] == -7.0).all()
    return host(q)[:M], host(d)[:M]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("act", [rf.GATE_SILU, rf.GATE_GELU])
def test_gate(M, K, act):
    announce("quantize_gated_acts", M, K, act)
    rng = np.random.default_rng(M + K)
    gu = (2.0 * rng.standard_normal((M, 2 * K))).astype(np.float32)
    ref = ff.gated(gu[:, :K], gu[:, K:], act == rf.GATE_GELU)
    both = to_dev(gu)
    q, d = run(both[:, :K], both[:, K:], act, M, K)               # two halves of one product
    assert_codes(q, d, ref)
    # codes and scales are those of the quantizer on the rounded values, but for values whose
    # rounding to fp32 hangs on the last bits of the fp64 arithmetic
    q2, d2 = oracle.quantize_acts(ref.astype(np.float32))
    assert np.array_equal(q, q2) and np.array_equal(d, d2)
    g2, u2 = both[:, :K].contiguous(), both[:, K:].contiguous()   # two products
    q3, d3 = run(g2, u2, act, M, K)
    assert np.array_equal(q, q3) and np.array_equal(d, d3)


def test_codes_at_the_least_alignment():
    """q and d 4 bytes off their allocations, at a size where codes are stored eight at a time."""
    announce("quantize_gated_acts, alignment")
    M, K = 1400, 1536
    gu = torch.randn(M, 2 * K, device=device(), generator=torch.Generator(device()).manual_seed(5))
    q, d = run(gu[:, :K], gu[:, K:], rf.GATE_SILU, M, K)
    q1, d1 = torch.zeros(M * K + 8, dtype=torch.int8, device=device()), torch.zeros(M * K // 32 + 2, device=device())
    rf.rfp2_quantize_gated_acts(gu[:, :K], gu[:, K:], M, K, rf.GATE_SILU, q1[4:-4], d1[1:-1])
    assert np.array_equal(host(q1)[4:-4], q.reshape(-1)) and not host(q1)[:4].any() and not host(q1)[-4:].any()
    assert np.array_equal(host(d1)[1:-1], d.reshape(-1)) and host(d1)[0] == 0 and host(d1)[-1] == 0
    out = empty((M, K), torch.float32)
    rf.rfp2_dequantize_acts(q1[4:-4], d1[1:-1], M, K, out)
    assert np.array_equal(host(out), (q.reshape(M, -1, 32).astype(np.float32) * d[..., None]).reshape(M, K))


@pytest.mark.parametrize("act", [rf.GATE_SILU, rf.GATE_GELU])
def test_range_of_the_gate(act):
    """From gates that vanish to gates that pass, with other halves that bring them back into
    range: silu(-100) is 4e-42 in fp32 and has three bits there; times 1e38 it has all of them."""
    announce("gate range", act)
    g = np.concatenate([np.linspace(-120, 120, 1024), -np.logspace(-30, 2, 512), np.logspace(-30, 20, 512),
                        -np.logspace(2, 30, 128)]).astype(np.float32)
    g = np.concatenate([g, np.zeros(-len(g) % 32, dtype=np.float32)])
    K = len(g)
    for size in (1.0, 1e-20, 1e18):
        u = np.full(K, size, dtype=np.float32)
        with np.errstate(over="ignore"):
            ref = ff.gated(g, u, act == rf.GATE_GELU)
        keep = np.abs(ref) < 1e38                                 # beyond: infinity in fp32, a NaN block
        u[~keep], ref[~keep] = 0.0, 0.0
        q, d = run(to_dev(g[None]), to_dev(u[None]), act, 1, K)
        assert_codes(q, d, ref[None])


@pytest.mark.parametrize("act", [rf.GATE_SILU, rf.GATE_GELU])
def test_infinities_and_nan(act):
    announce("gate of infinities", act)
    rng = np.random.default_rng(2)
    M, K = 5, 128
    g, u = rng.standard_normal((2, M, K)).astype(np.float32)
    g[0, 3], g[1, 40], g[2, 70], u[3, 127], u[4, 0] = np.nan, np.inf, -np.inf, np.nan, -np.inf
    q, d = run(to_dev(g), to_dev(u), act, M, K)
    ref = ff.gated(g, u, act == rf.GATE_GELU)
    for m, b in ((0, 0), (1, 1), (2, 2), (3, 3), (4, 0)):
        assert np.isnan(d[m, b]) and not q[m, 32 * b:32 * b + 32].any()
        rest = [i for i in range(4) if i != b]
        r = ref[m].reshape(4, 32)[rest].reshape(1, -1)
        assert_codes(q[m].reshape(4, 32)[rest].reshape(1, -1), d[m, rest][None], r)


@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (7, 5120), (1030, 4096), (1, 1 << 20)])
def test_values_of_codes(M, K):
    announce("dequantize_acts", M, K)
    rng = np.random.default_rng(M)
    a = (rng.standard_normal((M, K)) * np.exp(4 * rng.standard_normal((M, 1)))).astype(np.float32)
    q, d = empty((M, K), torch.int8), empty((M, K // 32), torch.float32)
    rf.rfp2_quantize_acts(to_dev(a), M, K, q, d)
    out = torch.full((M + 1, K), -7.0, device=device())
    rf.rfp2_dequantize_acts(q, d, M, K, out)
    want = host(q).reshape(M, K // 32, 32).astype(np.float32) * host(d)[..., None]
    assert np.array_equal(host(out)[:M], want.reshape(M, K)) and (host(out)[M] == -7.0).all()


def test_values_of_all_codes():
    announce("dequantize_acts, all codes")
    q = np.arange(-128, 128, dtype=np.int8).reshape(2, 128)
    d = np.array([[1.0, 2.0 ** -149, np.nan, -3.5], [0.0, np.inf, 1e30, 0.1]], dtype=np.float32)
    out = empty((2, 128), torch.float32)
    rf.rfp2_dequantize_acts(to_dev(q), to_dev(d), 2, 128, out)
    with np.errstate(invalid="ignore"):
        want = (q.reshape(2, 4, 32).astype(np.float32) * d[..., None]).reshape(2, 128)
    assert np.array_equal(host(out), want, equal_nan=True)


@pytest.mark.parametrize("seed", range(4))
def test_codes_of_any_values(seed):
    """Codes and scales without divisions are those of rfp2_quantize_acts bit for bit: 64 as the gate
    passes 64 times the other half exactly (exp(-64) is below half a step of fp64), whose values
    here have any exponent, subnormal scales and quotients close to the border of two codes among
    them."""
    announce("codes of any values", seed)
    rng = np.random.default_rng(seed)
    M, K = 1024, 4096
    u = (rng.integers(0, 1 << 23, (M, K), dtype=np.uint32) | np.uint32(127 << 23)).view(np.float32) - 1
    u = u * np.exp2(rng.integers(-150, 121, (M, K // 32, 1)).astype(np.float64)).repeat(32, -1).reshape(M, K)
    u *= np.exp2(-rng.integers(0, 12, (M, K)).astype(np.float64)) * rng.choice([-1.0, 1.0], (M, K))
    # every second row: multiples of a half of the block's scale, and their neighbours in fp32
    b = u[::2].reshape(-1, K // 32, 32).astype(np.float32)
    top = np.abs(b).max(-1, keepdims=True)
    d = np.where(top > 0, (top.astype(np.float64) / 127).astype(np.float32), np.float32(1))
    half = ((rng.integers(-127, 127, b.shape) + 0.5) * d.astype(np.float64)).astype(np.float32)
    half = np.where(rng.random(b.shape) < 0.5, half, np.nextafter(half, np.float32(0)))
    half[..., :1] = top
    u = u.astype(np.float32)
    u[::2] = half.reshape(-1, K)
    y = to_dev(u) * 64.0
    q, d = run(torch.full((M, K), 64.0, device=device()), to_dev(u), rf.GATE_SILU, M, K)
    q2, d2 = empty((M, K), torch.int8), empty((M, K // 32), torch.float32)
    rf.rfp2_quantize_acts(y, M, K, q2, d2)
    assert np.array_equal(d, host(d2), equal_nan=True) and np.array_equal(q, host(q2))
