"""GPU parity of the routing: ids equal the oracle's, weights within one rounding of the
fp64 arithmetic (2^-24 of the value; exp and the sums within 2^-40)."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, host, to_dev, torch
from oracle import feed_forward as ff

pytestmark = pytest.mark.gpu


def run(logits, bias, sigmoid, groups, group_top, top_groups, k, renorm, scale, gap=0):
    T, E = logits.shape
    wide = torch.full((T, E + gap), float("nan"), device=device())
    wide[:, :E] = to_dev(logits)
    ids = torch.full((T + 1, k), 12345, dtype=torch.int32, device=device())
    w = torch.full((T + 1, k), -7.0, device=device())
    err = torch.zeros(1, dtype=torch.int32, device=device())
    rf.rfp2_moe_route(wide, T, E, None if bias is None else to_dev(bias),
                      rf.ROUTE_SIGMOID if sigmoid else rf.ROUTE_SOFTMAX, groups, group_top, top_groups, k,
                      renorm, scale, ids, w, err)
    ids, w = host(ids), host(w)
    assert (ids[T] == 12345).all() and (w[T] == -7.0).all()
    return ids[:T], w[:T], int(host(err)[0])


def check(logits, bias, sigmoid, groups, group_top, top_groups, k, renorm, scale, gap=0):
    ids, w, err = run(logits, bias, sigmoid, groups, group_top, top_groups, k, renorm, scale, gap)
    assert err == 0
    for t in range(len(logits)):
        want, wref = ff.route(logits[t], bias, sigmoid, groups, group_top, top_groups, k, renorm, scale)
        assert ids[t].tolist() == want, (t, ids[t].tolist(), want)
        wref = np.array(wref)
        # half a step of the value and of the smallest numbers, and the fp64 arithmetic
        assert np.all(np.abs(w[t] - wref) <= (2.0 ** -24 + 2.0 ** -40) * np.abs(wref) + 2.0 ** -150), (t, w[t], wref)


# T, E, sigmoid, bias, groups, group_top, top_groups, top_k, renorm, scale, gap
CASES = [
    (1, 1, False, False, 1, 1, 1, 1, True, 1.0, 0), (1, 128, False, False, 1, 1, 1, 8, True, 1.0, 0),
    (3, 2, True, True, 1, 1, 1, 2, True, 1.0, 3), (17, 60, False, False, 1, 1, 1, 4, False, 1.0, 0),
    (5, 64, True, False, 1, 1, 1, 6, True, 2.5, 1), (130, 128, False, True, 1, 1, 1, 8, False, 0.5, 0),
    (33, 256, True, True, 8, 2, 4, 8, True, 2.5, 0), (9, 160, False, False, 8, 1, 3, 6, False, 16.0, 0),
    (7, 65, True, True, 5, 2, 2, 16, True, 1.0, 7), (4, 512, False, True, 64, 2, 9, 64, True, 1.0, 0),
    (2, 2048, True, True, 1, 1, 1, 64, True, 1.0, 0), (2, 2048, False, False, 32, 1, 5, 64, False, 1.0, 5),
    (3, 384, True, True, 1, 1, 1, 8, True, 2.5, 0), (3, 64, False, False, 64, 1, 8, 8, True, 1.0, 0),
    (6, 1000, False, False, 1, 1, 1, 10, True, 1.0, 1), (5, 2, False, True, 2, 1, 1, 1, True, 1.0, 0),
    (1100, 16, False, False, 1, 1, 1, 2, True, 1.0, 0), (700, 96, True, True, 4, 2, 2, 5, True, 1.0, 0),
    (11, 66, False, False, 1, 1, 1, 64, True, 1.0, 0), (3, 8, True, False, 1, 1, 1, 8, False, -1.0, 0),
]


@pytest.mark.parametrize("case", CASES)
def test_route(case):
    announce("moe_route", *case)
    T, E, sigmoid, bias, groups, group_top, top_groups, k, renorm, scale, gap = case
    rng = np.random.default_rng(T * 31 + E)
    l = (2.0 * rng.standard_normal((T, E))).astype(np.float32)
    b = (0.2 * rng.standard_normal(E)).astype(np.float32) if bias else None
    check(l, b, sigmoid, groups, group_top, top_groups, k, renorm, scale, gap)


@pytest.mark.parametrize("E,groups,k", [(64, 1, 8), (128, 8, 8), (200, 4, 16), (24, 1, 24)])
@pytest.mark.parametrize("sigmoid,bias", [(False, False), (True, True), (False, True)])
def test_equal_logits_go_to_the_lower_expert(E, groups, k, sigmoid, bias):
    announce("moe_route ties", E, groups, k, sigmoid, bias)
    rng = np.random.default_rng(E + k)
    l = rng.integers(-2, 3, (40, E)).astype(np.float32)          # five values: ties everywhere
    l[0] = 0.0
    l[1, ::2] = -0.0
    b = np.zeros(E, dtype=np.float32) if bias else None
    top_groups = max(1, groups // 2) if groups > 1 else 1
    check(l, b, sigmoid, groups, 1, top_groups, k, True, 1.0)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("bias,groups,group_top", [(False, 1, 1), (True, 1, 1), (True, 4, 2), (False, 4, 1)])
def test_masked_experts(sigmoid, bias, groups, group_top):
    announce("moe_route masks", sigmoid, bias, groups, group_top)
    E, k = 64, 6
    rng = np.random.default_rng(7)
    l = rng.standard_normal((24, E)).astype(np.float32)
    for t in range(24):                                         # from no expert masked to all of them
        l[t, rng.permutation(E)[:int(round(E * t / 23))]] = -np.inf
    l[5, 16:32] = -np.inf                                       # a whole group
    l[6, :48] = -np.inf                                         # three
    l[7] = -np.inf
    l[7, 40] = 1.0                                              # one expert left
    l[8] = np.finfo(np.float32).min                             # the lowest number is no mask
    b = (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None
    check(l, b, sigmoid, groups, group_top, 2 if groups > 1 else 1, k, True, 1.0)
    ids, w, _ = run(l, b, sigmoid, groups, group_top, 2 if groups > 1 else 1, k, True, 1.0)
    assert not w[23].any() and ids[23].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [8, 128, 300])
def test_what_cannot_be_routed_is_loud(sigmoid, E):
    announce("moe_route NaN", sigmoid, E)
    rng = np.random.default_rng(E)
    l = rng.standard_normal((9, E)).astype(np.float32)
    l[2, E - 1] = np.nan
    l[4, 0] = np.inf
    l[6, 3] = -np.inf                                           # a mask is fine
    ids, w, err = run(l, None, sigmoid, 1, 1, 1, 4, True, 1.0)
    assert err == 1
    for t in range(9):
        if t in (2, 4):
            assert (ids[t] == -1).all() and np.isnan(w[t]).all()
        else:
            assert ids[t].tolist() == ff.route(l[t], None, sigmoid, 1, 1, 1, 4, True, 1.0)[0]
    for value in (np.nan, np.inf, -np.inf):
        b = np.zeros(E, dtype=np.float32)
        b[E // 2] = value
        ids, w, err = run(l[:1], b, sigmoid, 1, 1, 1, 4, True, 1.0)
        assert err == 1 and (ids == -1).all() and np.isnan(w).all()


def test_far_logits():
    """Scores that underflow: chosen by their logits all the same, weight 0."""
    announce("moe_route far logits")
    l = np.full((2, 70), -3e38, dtype=np.float32)
    l[0, 3], l[0, 50], l[0, 60] = 3e38, -1e30, -1e31
    l[1, 69], l[1, 1] = -5000.0, -4000.0
    for sigmoid in (False, True):
        check(l, None, sigmoid, 1, 1, 1, 3, True, 1.0)
    # neighbours in fp32 stay apart with a bias that is larger than both
    l = np.zeros((1, 128), dtype=np.float32)
    l[0] = 0.25
    l[0, 100] = np.nextafter(np.float32(0.25), np.float32(1))
    check(l, np.full(128, 100.0, dtype=np.float32), True, 1, 1, 1, 2, True, 1.0)


def test_without_err():
    announce("moe_route without err")
    l = to_dev(np.array([[np.nan, 1.0], [1.0, 0.0]], dtype=np.float32))
    ids, w = torch.zeros(2, 1, dtype=torch.int32, device=device()), torch.zeros(2, 1, device=device())
    rf.rfp2_moe_route(l, 2, 2, None, rf.ROUTE_SOFTMAX, 1, 1, 1, 1, True, 1.0, ids, w)
    assert host(ids).tolist() == [[-1], [0]] and np.isnan(host(w)[0, 0]) and host(w)[1, 0] == 1.0
