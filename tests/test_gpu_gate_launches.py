"""The gate call beyond the values that one launch holds: 2^31 pieces of four."""
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [rf.GATE_SILU, rf.GATE_GELU])
def test_more_pieces_than_a_launch_holds(act):
    """gate and up are the same 32 GiB, the same 4096 rows again and again but for some around
    the border of the launches and at the ends; codes 4 bytes off are stored four at a time."""
    announce("gate, 2^31 pieces", act)
    K, many = 4096, 4096
    border = ((1 << 31) - 512) // (K // 4)      # rows of a launch
    M = border + 5

    def normal(*shape, seed):
        return torch.randn(*shape, generator=torch.Generator(device()).manual_seed(seed), device=device())

    def few(x):
        n = len(x)
        q, d = torch.empty(n, K, dtype=torch.int8, device=device()), torch.empty(n, K // 32, device=device())
        rf.rfp2_quantize_gated_acts(x, x, n, K, act, q, d)
        return q, d

    base = normal(many, K, seed=1)
    at = [0, 1, M // 2, border - 1, border, border + 1, M - 1]
    other = 3.0 * normal(len(at), K, seed=2)
    x = torch.empty(M, K, device=device())
    for m in range(0, M, many):
        x[m:m + many] = base[:M - m]
    for i, r in enumerate(at):
        x[r] = other[i]
    q = torch.full((M * K + 8,), 99, dtype=torch.int8, device=device())
    d = torch.full((M * K // 32 + 2,), -7.0, device=device())
    rf.rfp2_quantize_gated_acts(x, x, M, K, act, q[4:-4], d[1:-1])
    assert bool((q[:4] == 99).all()) and bool((q[-4:] == 99).all()) and d[0] == -7.0 and d[-1] == -7.0
    qr, dr = q[4:-4].view(M, K), d[1:-1].view(M, K // 32)
    q1, d1 = few(other)
    for i, r in enumerate(at):
        assert torch.equal(qr[r], q1[i]) and torch.equal(dr[r], d1[i]), r
    q2, d2 = few(base)
    q3, d3 = torch.empty_like(q2), torch.empty_like(d2)
    for m in range(0, M, many):
        n = min(many, M - m)
        q3.copy_(q2)
        d3.copy_(d2)
        for i, r in enumerate(at):
            if m <= r < m + n:
                q3[r - m], d3[r - m] = q1[i], d1[i]
        assert torch.equal(qr[m:m + n], q3[:n]) and torch.equal(dr[m:m + n], d3[:n]), m
