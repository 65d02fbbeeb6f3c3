"""GPU parity of the routing's renormalised weights where the chosen scores are far below
one, against the definition in decimals."""
import numpy as np
import pytest

import _far_scores as far
import bit_gemv_amd as rf
from _gpu import announce, device, host, to_dev, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 1027])
@pytest.mark.parametrize("case", far.cases(), ids=lambda c: c[0])
def test_weights_of_far_scores(case, tokens):
    name, l, bias, sigmoid, groups, group_top, top_groups, k, scale, chosen = case
    announce("moe_route far scores", name, tokens)
    E = len(l)
    rng = np.random.default_rng(E)
    logits = rng.standard_normal((tokens, E)).astype(np.float32)      # among tokens of everyday scores
    logits[-1] = l
    ids = torch.zeros(tokens, k, dtype=torch.int32, device=device())
    w = torch.zeros(tokens, k, device=device())
    err = torch.zeros(1, dtype=torch.int32, device=device())
    rf.rfp2_moe_route(to_dev(logits), tokens, E, None if bias is None else to_dev(bias),
                      rf.ROUTE_SIGMOID if sigmoid else rf.ROUTE_SOFTMAX, groups, group_top, top_groups, k,
                      True, scale, ids, w, err)
    assert int(host(err)[0]) == 0 and host(ids)[-1].tolist() == chosen
    want = np.array(far.weights(l, chosen, sigmoid, scale))
    # one rounding to fp32, of the smallest numbers too, and the fp64 arithmetic
    assert np.all(np.abs(host(w)[-1] - want) <= (2.0 ** -24 + 2.0 ** -40) * want + 2.0 ** -150), (host(w)[-1], want)
    if tokens > 1:
        assert np.abs(host(w)[:-1].sum(-1) - scale).max() <= (k + 1) * 2.0 ** -24 * scale
