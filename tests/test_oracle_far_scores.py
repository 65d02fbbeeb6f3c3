"""The oracle's renormalised weights where the chosen scores are far below one (CPU only)."""
import numpy as np
import pytest

import _far_scores as far
from oracle import feed_forward as ff


@pytest.mark.parametrize("case", far.cases(), ids=lambda c: c[0])
def test_weights_of_far_scores(case):
    _, l, bias, sigmoid, groups, group_top, top_groups, k, scale, chosen = case
    ids, w = ff.route(l, bias, sigmoid, groups, group_top, top_groups, k, True, scale)
    assert ids == chosen
    # a score 1 / (1 + e^-l) or e^(l - top), the sum and the quotient: some ten roundings, and
    # the library's exponentials within a step
    assert np.allclose(w, far.weights(l, ids, sigmoid, scale), rtol=2.0 ** -48, atol=0.0)
