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


def test_in_place_with_two_strides():
    """Refused for the strides and nothing else: the same calls with one stride fail later, on an address."""
    lib = gq.load()
    rope = gq.gqa_rope_init(64)
    r = ctypes.addressof(rope)

    def turn(qs, qos, at=256, positions=768):
        return lib.gqa_rope(r, at, None, positions, at, None, 4, 8, 0, 64, qs, 0, qos, 0, 0, None)

    def append(qs, qos, v=768):
        return lib.gqa_append_paged(r, 256, 512, v, 256, 1024, 1280, 1536, 1552, 1568, 4, 2, 8, 2, 64, qs, 128, 128, qos,
                                    16, 4, 4, None)

    assert turn(512, 640) == gq.GQA_ERR_INVALID_ARG and turn(640, 512) == gq.GQA_ERR_INVALID_ARG
    assert turn(512, 512, at=264) == gq.GQA_ERR_MISALIGNED
    assert append(512, 640) == gq.GQA_ERR_INVALID_ARG
    assert append(512, 512, v=776) == gq.GQA_ERR_MISALIGNED
