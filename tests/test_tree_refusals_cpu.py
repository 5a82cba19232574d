"""Refusals of the calls over trees and of the rotary calls, before any CUDA call: addresses and strides."""
import ctypes

import pytest

from tests.test_paged_cpu import FAKE, INVALID
from tests.test_tree_cpu import attention, decode, gdn, maps, rotary, side  # noqa: F401

OFF = ctypes.c_void_p(0x10004)  # a multiple of 4 bytes, but not of 8


@pytest.mark.parametrize("off", [OFF, ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10002)])
def test_words_of_eight_bytes_off_their_boundary(gdn, off):  # noqa: F811
    assert maps(gdn, masks=off) == INVALID
    assert attention(gdn, masks=off) == INVALID
    assert decode(gdn, masks=off) == INVALID
    assert rotary(gdn, freq=off) == INVALID
