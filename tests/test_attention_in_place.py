"""The fused rotation and write refuses an output that is one of its inputs (no GPU,
nothing is launched): a lane reads its pair's other value while others write theirs."""
import pytest

from test_attention_host import P, SHAPE, cache, fused


@pytest.mark.parametrize("inputs", [dict(q=P), dict(k=P), dict(v=P), dict(q=P, k=P, v=P)])
def test_the_output_is_none_of_the_inputs(inputs):
    args = dict(q=2 * P, k=3 * P, v=4 * P, out=P)
    args.update(inputs)
    # every other argument is in order: with a good output the call would be launched
    assert fused(cache(), **args) == SHAPE
