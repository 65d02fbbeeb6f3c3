"""GPU parity of the routing's forms that prompts take, several tokens a workgroup with
its last one partly filled, and of more than 512 experts: each count of experts a lane, with
and without scores and groups in LDS."""
import numpy as np
import pytest

from _gpu import announce
from test_gpu_moe_route import check

pytestmark = pytest.mark.gpu

# T, E, sigmoid, bias, groups, group_top, top_groups, top_k, renorm, scale, gap
CASES = [
    # nothing in LDS
    (1025, 128, False, False, 1, 1, 1, 8, True, 1.0, 0), (1027, 200, True, False, 1, 1, 1, 8, False, 2.5, 1),
    (1026, 512, True, False, 1, 1, 1, 10, True, 1.0, 0), (1025, 320, False, False, 1, 1, 1, 16, True, 1.0, 0),
    # scores
    (1025, 128, False, False, 1, 1, 1, 8, False, 1.0, 0), (1026, 255, False, True, 1, 1, 1, 8, True, 1.0, 0),
    (1027, 512, False, False, 1, 1, 1, 6, False, 1.0, 0), (1025, 384, True, True, 1, 1, 1, 8, True, 2.5, 3),
    # what groups are compared by
    (1025, 160, False, False, 8, 1, 3, 6, True, 1.0, 0), (1026, 96, True, False, 4, 1, 2, 6, True, 1.0, 0),
    (1027, 512, True, False, 16, 1, 5, 8, False, 1.0, 0), (1030, 60, True, False, 5, 1, 2, 4, True, 1.0, 0),
    # both, up to 32 KiB a workgroup
    (1027, 160, False, False, 8, 1, 3, 6, False, 1.0, 0), (1025, 100, False, False, 4, 1, 2, 6, False, 16.0, 0),
    (1030, 60, True, True, 4, 2, 2, 5, True, 1.0, 1), (1025, 128, True, True, 8, 2, 4, 8, True, 2.5, 0),
    (1026, 256, True, True, 8, 2, 4, 8, True, 2.5, 3), (1027, 512, False, True, 64, 2, 9, 16, True, 1.0, 0),
    (1025, 512, False, False, 32, 1, 4, 12, False, 1.0, 0),
    # 513 to 1024 experts, and up to 2048, with a bias
    (5, 600, True, True, 1, 1, 1, 8, True, 1.0, 0), (4, 600, False, True, 8, 2, 3, 16, False, 1.0, 1),
    (3, 1000, False, True, 1, 1, 1, 64, True, 1.0, 0), (4, 1000, True, True, 8, 2, 4, 10, True, 2.5, 0),
    (3, 1024, False, True, 64, 2, 9, 64, True, 1.0, 0), (2, 513, True, True, 1, 1, 1, 64, True, 1.0, 0),
    (3, 2048, False, True, 32, 2, 5, 64, True, 1.0, 0), (2, 1025, True, True, 5, 2, 2, 30, False, 1.0, 0),
    (1031, 700, True, True, 7, 2, 3, 8, True, 1.0, 0),
]


@pytest.mark.parametrize("case", CASES)
def test_route(case):
    announce("moe_route forms", *case)
    T, E, sigmoid, bias, groups, group_top, top_groups, k, renorm, scale, gap = case
    rng = np.random.default_rng(T * 37 + E)
    l = (2.0 * rng.standard_normal((T, E))).astype(np.float32)
    l[T // 2] = -np.inf                                         # a token without experts among the others
    l[T - 1, 1::3] = -np.inf
    b = (0.2 * rng.standard_normal(E)).astype(np.float32) if bias else None
    check(l, b, sigmoid, groups, group_top, top_groups, k, renorm, scale, gap)
