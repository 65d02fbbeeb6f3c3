"""Values written over the codes or scales they come from are refused (no GPU, nothing is
launched): four bytes a value would overwrite codes that others still read."""
import pytest

import bit_gemv_amd as rf

M, K = 2, 64
Q, D, A = 0x10000, 0x20000, 0x30000           # aligned fake device addresses: never dereferenced


@pytest.mark.parametrize("q,d", [
    (A, D), (Q, A), (A + 4 * M * K - 4, D), (A - M * K + 4, D), (Q, A + 4 * M * K - 4),
    (Q, A - M * K // 8 + 4), (A + 16, A + 32),
])
def test_values_over_their_codes(q, d):
    assert rf.lib().rfp2_dequantize_acts(q, d, M, K, A, None) == rf.RFP2_E_SHAPE
