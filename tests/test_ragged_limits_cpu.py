"""Refusals at the ends of what a packed batch's arguments can hold, without a GPU."""
import ctypes

import pytest

import grouped_query_decode_gb300 as gq
from test_ragged_cpu import packed, paged

INT_MAX = (1 << 31) - 1


@pytest.mark.parametrize("call", [packed, paged])
def test_scales_whose_base_2_form_overflows(call):
    """Scores are scaled by scale * log2(e): 2.36e38 is the last scale for which that is finite."""
    lib = gq.load()
    for bad in (2.4e38, 3.0e38, 3.4e38):
        assert call(lib, scale=bad) == gq.GQA_ERR_INVALID_ARG, bad
    # what is wrong behind the scale is seen behind it
    for good in (1e-45, 1.0, 2.3e38):
        assert call(lib, scale=good, out=1288) == gq.GQA_ERR_MISALIGNED, good
