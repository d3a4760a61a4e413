"""Refusals of the target's side of a step at the ends of its arguments' ranges: nothing is launched, so
these run without a GPU."""
import math

from test_target_abi import INVALID, OK, attend


def test_attention_of_scales_at_the_end_of_fp32():
    """Scores are formed times scale log2(e): a scale for which that is infinite makes a score of 0 NaN."""
    nothing = dict(B=0, rows=0, pages=None, lengths=None, q=None, out=None)
    most = (2.0 ** 128 - 2.0 ** 103) * math.log(2.0)            # what rounds to the largest number
    assert attend(**nothing, scale=most * (1 - 2.0 ** -20)) == OK
    for scale in (most * (1 + 2.0 ** -20), 3.0e38, (2.0 - 2.0 ** -23) * 2.0 ** 127):
        assert attend(**nothing, scale=scale) == INVALID, scale
    assert attend(**nothing, scale=2.0 ** -149) == OK
