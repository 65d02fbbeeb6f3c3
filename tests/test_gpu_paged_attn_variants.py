"""Every variant of the attention: all head sizes, all counts of query rows to a
key/value head that pick another kernel, both formats; the join by waves at every head
size; decided winners among scores of more than a thousand; the range of an int8 cache.
Tolerances are those of test_gpu_paged_attn but where a test derives its own."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, host, to_dev, torch
from oracle import attention as oa
from test_gpu_paged_attn import F16, I8, Setup, assert_close

pytestmark = pytest.mark.gpu

DIMS = [32, 64, 96, 128, 160, 192, 224, 256]
# new tokens and query heads to a key/value head: 1 to 16 rows on one wave, to 32 on two,
# to 64 on four, more as further items (the last of them with 1 and with 16 rows)
ROWS = [(1, 1), (1, 4), (2, 4), (1, 7), (1, 12), (4, 4), (3, 7), (4, 8), (5, 8), (6, 8), (7, 9),
        (8, 8), (5, 13), (8, 10)]


@pytest.mark.parametrize("fmt", [F16, I8])
@pytest.mark.parametrize("T,group", ROWS)
@pytest.mark.parametrize("D", DIMS)
def test_rows_and_heads(fmt, T, group, D):
    """Ragged, one sequence of them long enough to be split over workgroups."""
    announce("paged_attn variant", fmt, T, group, D)
    s = Setup(fmt, [3, 331, 0, 60], T, group, 1, D, 16, seed=T * 1000 + group * 10 + D)
    err = torch.zeros(1, dtype=torch.int32, device=device())
    assert_close(host(s.run(err=err)), *s.reference())
    assert int(host(err)[0]) == 0
    assert_close(host(s.run(45)), *s.reference(45))


@pytest.mark.parametrize("fmt", [F16, I8])
@pytest.mark.parametrize("T,H,Hkv", [(1, 8, 4), (3, 6, 2)])
@pytest.mark.parametrize("D", DIMS)
def test_join_by_waves(fmt, D, T, H, Hkv):
    """More than 256 output rows, most of whose items lie in two or more shares."""
    announce("paged_attn join by waves", fmt, D, T, H, Hkv)
    rng = np.random.default_rng(D)
    lens = [0, 900] + rng.integers(1, 400, 39).tolist()
    s = Setup(fmt, lens, T, H, Hkv, D, 32, seed=D + T)
    assert len(lens) * T * H > 256
    assert_close(host(s.run()), *s.reference())


@pytest.mark.parametrize("fmt", [F16, I8])
@pytest.mark.parametrize("D", [64, 96, 256])
def test_decided_winners_among_large_scores(fmt, D):
    """Each row has one token whose score is ahead of all others by more than 160 in base
    2, so that every other weight is below fp32's smallest: the result is that token's
    value.  Scores pass a thousand and grow towards the winners.

    Weights and their sum are scaled by the same numbers (2^(m - m') with m the running
    maximum), each product rounded: a few of them until the winner is met and at most one
    after it a wave and share; the weight times the value's scale, times the value, the
    reciprocal of the sum and its product are four more: 16 * 2^-24 holds them."""
    announce("paged_attn winners", fmt, D)
    n, H = 700, 4
    s = Setup(fmt, [n, 40], 1, H, 1, D, 16, seed=D)
    rng = np.random.default_rng(D)
    q = rng.choice([-1.0, 1.0], (2, 1, H, D)).astype(np.float32)
    at = np.array([[0, 63, 450, n - 1], [39, 1, 32, 0]])
    for b, m in enumerate((n, 40)):
        k = rng.integers(-1, 2, (m, 1, D)).astype(np.float32)
        k[:, 0] += 0.4 * np.linspace(-1, 1, m)[:, None] * q[b, 0, 3]   # rising for the last head
        for h in range(H):
            k[at[b, h], 0] = 3 * q[b, 0, h]
        v = rng.standard_normal((m, 1, D)).astype(np.float32)
        seq, pos = np.full(m, b, np.int32), np.arange(m, dtype=np.int32)
        rf.rfp2_kv_write(s.cache, to_dev(k), to_dev(v), m, to_dev(seq), to_dev(pos))
        s.k[b], s.v[b] = oa.held(k, fmt == I8), oa.held(v, fmt == I8)
    s.q, s.scale = q, 16.0
    got = host(s.run())
    for b in range(2):
        for h in range(H):
            score = 16.0 * (s.k[b][:, 0] @ q[b, 0, h].astype(np.float64))
            second, first = np.sort(score)[-2:]
            assert score.argmax() == at[b, h] and first > 1000 and (first - second) * 1.4427 > 160
            value = s.v[b][at[b, h], 0]
            err = np.abs(got[b, 0, h] - value)
            assert np.all(err <= 16 * 2.0 ** -24 * np.abs(value)), (b, h, err.max())
            other = s.v[b][(at[b, h] + 1) % len(s.v[b]), 0]
            # (the bound rejects the neighbour's value, and zeros)
            assert (np.abs(other - value) > 16 * 2.0 ** -24 * np.abs(value)).mean() > 0.9


def test_range_of_an_int8_cache():
    """Keys of 2^104 against queries of 2^-104, values of 2^87."""
    announce("paged_attn int8 range")
    n, D = 300, 128
    s = Setup(I8, [n], 1, 4, 1, D, 16, seed=20)
    rng = np.random.default_rng(20)
    k, v = rng.uniform(-1, 1, (2, n, 1, D)).astype(np.float32)
    k, v = (k * 2.0 ** 104).astype(np.float32), (v * 2.0 ** 87).astype(np.float32)
    s.q = (s.q * 2.0 ** -104).astype(np.float32)
    rf.rfp2_kv_write(s.cache, to_dev(k), to_dev(v), n, to_dev(np.zeros(n, np.int32)),
                     to_dev(np.arange(n, dtype=np.int32)))
    s.k, s.v = [oa.held(k, True)], [oa.held(v, True)]
    assert_close(host(s.run()), *s.reference())


@pytest.mark.parametrize("fmt", [F16, I8])
@pytest.mark.parametrize("lens,T,H,Hkv", [([300], 1, 1024, 1024), ([300], 1, 600, 600), ([70], 8, 1024, 512),
                                          ([40, 0, 9], 1, 1024, 1024)])
def test_many_heads(fmt, lens, T, H, Hkv):
    """As many (sequence, head) items as there are workgroups, and more of one sequence."""
    announce("paged_attn many heads", fmt, lens, T, H, Hkv)
    s = Setup(fmt, lens, T, H, Hkv, 32, 8, seed=H + T)
    assert_close(host(s.run()), *s.reference())


@pytest.mark.parametrize("fmt", [F16, I8])
def test_first_sequences_of_a_larger_buffer(fmt):
    """B below the cache's sequences, queries q[:B] of a buffer for all of them."""
    announce("paged_attn part of a buffer", fmt)
    s = Setup(fmt, [90, 33, 150, 20], 3, 4, 2, 64, 16, seed=21)
    ref, tol = s.reference()
    q = to_dev(s.q)
    lens = to_dev(np.array(s.lens, np.int32))
    y = torch.full((4, 3, 4, 64), -3.0, device=device())
    rf.rfp2_paged_attn(s.cache, q[:2], 2, 3, 4, lens, s.scale, y)
    got = host(y)
    assert_close(got[:2], ref[:2], tol[:2])
    assert (got[2:] == -3.0).all()
