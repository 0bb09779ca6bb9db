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


def test_append_to_more_sequences_than_the_search_can_count():
    """The search for a token's sequence steps through B + 1 offsets, 32 at a time, in 32 bits."""
    lib = gq.load()
    rope = gq.gqa_rope_init(64)

    def call(B, kp=1024):
        return lib.gqa_append_paged(ctypes.addressof(rope), None, 512, 768, None, kp, 1280, 1536, 1552, 1568, 4, B, 0, 2, 64, 0, 128, 128,
                                    0, 16, 4, 4, None)

    for B in (INT_MAX, INT_MAX - 1, INT_MAX - 32):
        assert call(B) == gq.GQA_ERR_UNSUPPORTED, B
    assert call(INT_MAX - 33, kp=1032) == gq.GQA_ERR_MISALIGNED
