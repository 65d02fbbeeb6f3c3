"""GPU parity of the gate's codes over many values: those of the quantizer on the fp32 values,
where every value of a block rounds to one fp32 number whichever way an error of 2^-43 of it
goes; between those of its two neighbours elsewhere."""
import numpy as np
import pytest

import bit_gemv_amd as rf
import oracle
from _gpu import announce, device, host, to_dev, torch
from oracle import feed_forward as ff

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [rf.GATE_SILU, rf.GATE_GELU])
@pytest.mark.parametrize("M,K", [(2048, 1536), (300, 4096)])
def test_codes(act, M, K):
    announce("gate rounding", act, M, K)
    rng = np.random.default_rng(M + act)
    g, u = (2.0 * rng.standard_normal((2, M, K))).astype(np.float32)
    q, d = torch.empty(M, K, dtype=torch.int8, device=device()), torch.empty(M, K // 32, device=device())
    rf.rfp2_quantize_gated_acts(to_dev(g), to_dev(u), M, K, act, q, d)
    q, d = host(q).reshape(M, -1, 32).astype(int), host(d)
    ref = ff.gated(g, u, act == rf.GATE_GELU)
    near, far = (ref * (1 - 2.0 ** -43)).astype(np.float32), (ref * (1 + 2.0 ** -43)).astype(np.float32)
    q0, d0 = oracle.quantize_acts(near)
    q1, d1 = oracle.quantize_acts(far)
    q0, q1 = q0.reshape(M, -1, 32).astype(int), q1.reshape(M, -1, 32).astype(int)
    one = (near == far).reshape(M, -1, 32).all(-1)
    assert one.mean() > 0.99                        # 32 * 2^-18 of the blocks are expected to be others
    assert np.array_equal(q[one], q0[one]) and np.array_equal(d[one], d0[one])
    assert np.all((d[~one] >= d0[~one]) & (d[~one] <= d1[~one]))
    # a larger scale lowers the code's magnitude: by a step at most, like a value's own neighbour
    a, b = np.minimum(q0, q1)[~one] - 1, np.maximum(q0, q1)[~one] + 1
    assert np.all((q[~one] >= a) & (q[~one] <= b))
