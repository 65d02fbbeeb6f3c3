"""Norms of rows that go past the caches, narrow and beyond what a thread keeps in registers, with
each of their outputs alone and together: the bits of small calls."""
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, torch

pytestmark = pytest.mark.gpu
EPS = 1e-5


def normal(*shape, seed=1):
    return torch.randn(*shape, generator=torch.Generator(device()).manual_seed(seed), device=device())


# what is written: h, y, codes; "x" and "add": y over that input
OUTPUTS = [(True, False, True), (True, True, False), (True, True, True), (False, True, True),
           (False, True, False), (False, False, True), (False, "x", True), (False, "add", True)]


@pytest.mark.parametrize("mode", ["row", "add", "sum"])
@pytest.mark.parametrize("K,values", [(4096, 1 << 20), (4096, 1 << 24), (16416, 1 << 20), (32768, 1 << 24),
                                      (131072, 1 << 24)])
def test_outputs_past_the_caches(mode, K, values):
    announce("norms past the caches, outputs", mode, K, values)
    T, k = values // K + 3, 2
    source, gain = normal(T, K), normal(K, seed=2)
    other = normal(T, K, seed=3) if mode == "add" else normal(T, k, K, seed=3)
    w = normal(T, k, seed=4)
    at = [0, T // 2, T - 1]

    def call(x, a, weights, h, y, q, d):
        n = len(x)
        if mode == "sum":
            rf.rfp2_moe_combine(x, a, weights, n, k, K, h, gain, EPS, y, q, d)
        else:
            rf.rfp2_add_rms_norm(x, a if mode == "add" else None, n, K, gain, EPS, h, y, q, d)

    def outputs(n, h, y, codes, x, a):
        return (torch.full((n, K), 7.0, device=device()) if h else None,
                x if y == "x" else a if y == "add" else torch.full((n, K), 7.0, device=device()) if y else None,
                torch.full((n, K), 99, dtype=torch.int8, device=device()) if codes else None,
                torch.full((n, K // 32), 7.0, device=device()) if codes else None)

    for h, y, codes in OUTPUTS:
        if (h and mode == "row") or (y == "add" and mode != "add"):
            continue
        x, a = source.clone(), other.clone()
        xs, as_ = x[at], a[at]
        many, few = outputs(T, h, y, codes, x, a), outputs(3, h, y, codes, xs, as_)
        call(x, a, w, *many)
        call(xs, as_, w[at], *few)
        for m, f in zip(many, few):
            assert m is None or torch.equal(m[at], f), (h, y, codes)
