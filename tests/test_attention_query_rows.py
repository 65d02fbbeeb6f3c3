"""How the binding finds the attention's query rows in a tensor (no GPU: shapes only)."""
import pytest

import bit_gemv_amd as rf

torch = pytest.importorskip("torch")


class FakeCache(rf.KvCache):
    head_dim = 64

    def __init__(self):
        self._struct = rf._KvCacheStruct()


def call(q, B, T, H):
    """The binding's own checks: the first that concerns q's rows raises before q's place is looked at."""
    rf.rfp2_paged_attn(FakeCache(), q, B, T, H, None, 0.1, None, workspace=object())


@pytest.mark.parametrize("shape", [(16, 2, 8, 64), (16, 2, 512), (9, 2, 512), (64, 2, 8, 64), (16, 2, 520)])
def test_a_buffer_of_more_sequences_is_refused(shape):
    """[more than B, new tokens, H * D ...] is neither of the two forms: taken as rows, its
    first B * new tokens rows would be the first token of twice as many sequences."""
    with pytest.raises(ValueError, match=r"q\[:8\]"):
        call(torch.zeros(shape), 8, 2, 8)


@pytest.mark.parametrize("shape,B,T,H", [
    ((8, 2, 8, 64), 8, 2, 8), ((8, 2, 512), 8, 2, 8),            # [B, new tokens, ...]
    ((16, 8, 64), 8, 2, 8), ((16, 512), 8, 2, 8), ((20, 512), 8, 2, 8), ((16, 2, 64), 8, 2, 2),
    ((20, 2, 64), 8, 2, 2),                                      # rows, H the number of new tokens
    ((1, 5, 512), 1, 5, 8), ((8, 1, 512), 8, 1, 8), ((16, 1, 512), 8, 1, 8), ((16, 512), 8, 1, 8),
])
def test_both_forms_reach_the_check_of_the_device(shape, B, T, H):
    with pytest.raises(ValueError, match="GPU"):
        call(torch.zeros(shape), B, T, H)


def test_a_cache_that_is_none_is_a_type_error():
    z = torch.zeros(2, 64)
    for call_it in (lambda c: rf.rfp2_kv_write(c, z, z, 2, z, z),
                    lambda c: rf.rfp2_rope_kv_write(c, z, z, z, 2, 1, z, z, z, 64, 0, 1.0, z),
                    lambda c: rf.rfp2_kv_read(c, 2, z, z, z, z),
                    lambda c: rf.rfp2_paged_attn(c, z, 2, 1, 1, z, 0.1, z),
                    lambda c: rf.rfp2_paged_attn_workspace_bytes(c, 2, 1, 1)):
        for c in (None, z):
            with pytest.raises(TypeError, match="KvCache"):
                call_it(c)
