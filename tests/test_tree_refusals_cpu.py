"""Refusals of the calls over trees and of the rotary calls, before any CUDA call: addresses and strides."""
import ctypes

import pytest
import torch

from tests.test_paged_cpu import INVALID, UNSUPPORTED
from tests.test_tree_cpu import attention, decode, gdn, maps, rotary, side  # noqa: F401

OFF = ctypes.c_void_p(0x10004)  # a multiple of 4 bytes, but not of 8


@pytest.mark.parametrize("off", [OFF, ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10002)])
def test_words_of_eight_bytes_off_their_boundary(gdn, off):  # noqa: F811
    assert maps(gdn, masks=off) == INVALID
    assert attention(gdn, masks=off) == INVALID
    assert decode(gdn, masks=off) == INVALID
    assert rotary(gdn, freq=off) == INVALID


ROWS = dict(T=4, d=128, rot=64)  # four tokens of four heads


@pytest.mark.parametrize("fields", [
    dict(ot=128, oh=128), dict(ot=256, oh=128), dict(ot=511, oh=128), dict(ot=128, oh=511), dict(ot=200, oh=300),
    dict(ot=130, oh=260), dict(x=0x20000, xt=256, xh=128, ot=256, oh=128), dict(ot=384, oh=256),
    dict(ot=(1 << 39) - 100, oh=1 << 39)])
def test_rotary_outputs_that_share_elements(gdn, fields):  # noqa: F811
    assert rotary(gdn, **ROWS, **fields) == INVALID
    assert rotary(gdn, **ROWS, q=side(gdn, heads=0), k=side(gdn, **fields)) == INVALID


@pytest.mark.parametrize("in_place", [False, True])
def test_rotary_outputs_by_their_elements(gdn, in_place):  # noqa: F811
    # every small shape: refused if and only if two rows share an element.  (q's side is looked at first; k's is one that
    # is turned down with another status, so that no call goes on.)
    from itertools import product
    d = 4
    for T, heads, ot, oh in product((1, 2, 3, 5), (1, 2, 3, 4), range(d, 26), range(d, 26)):
        at = [t * ot + h * oh + i for t in range(T) for h in range(heads) for i in range(d)]
        strides = dict(xt=ot, xh=oh) if in_place else dict(xt=d * heads, xh=d)
        got = rotary(gdn, T=T, d=d, rot=2, k=side(gdn, heads=1 << 17), x=0x20000 if in_place else 0x10000, heads=heads,
                     ot=ot, oh=oh, **strides)
        assert got == (UNSUPPORTED if len(set(at)) == len(at) else INVALID), (T, heads, ot, oh)


def test_rotary_outputs_far_apart(gdn):  # noqa: F811
    big, most = 1 << 39, (1 << 31) - 1
    for T, heads, ot, oh, status in [
            (most, 65536, 128 * 65536, 128, UNSUPPORTED), (most, 65536, 128, big - 128, UNSUPPORTED),
            (most, 2, 128, 128 * most - 1, INVALID), (most, 65536, big, big, INVALID), (2, 65536, big, 128, UNSUPPORTED),
            (2, 65536, big, 1 << 25, INVALID)]:
        got = rotary(gdn, T=T, d=128, rot=64, k=side(gdn, heads=1 << 17), heads=heads, ot=ot, oh=oh)
        assert got == status, (T, heads, ot, oh)


@pytest.mark.parametrize("rot", [2, 16, 128])
@pytest.mark.parametrize("length,fast,slow", [(4, 32.0, 1.0), (1, 32.0, 1.0), (4096, 5000.0, 1000.0), (4096, 1000.0, 1000.0),
                                              (6, 1.0, 1.0), (4096, 32.0, 1.0), (1 << 40, 0.001, 0.0001)])
def test_yarn_pairs_outside_its_ramp(gdn, rot, length, fast, slow):  # noqa: F811
    # a pair that turns less than `slow` times over the length is divided by the factor, one that turns more than `fast`
    # times stays; what lies between is between
    from math import pi
    got = gdn.gdn_rotary_frequencies(rot, 1e4, "yarn", 8.0, length, fast, slow).tolist()
    plain = gdn.gdn_rotary_frequencies(rot, 1e4).tolist()
    for i, (f, p) in enumerate(zip(got, plain)):
        turns = length * 1e4 ** (-2 * i / rot) / (2 * pi)
        if turns < slow * (1 - 1e-9):
            assert abs(f - p / 8) <= p / 8 * 2.0 ** -45 + 1, i
        elif turns > fast * (1 + 1e-9):
            assert abs(f - p) <= p * 2.0 ** -45 + 1, i
        else:
            assert p / 8 * (1 - 2.0 ** -45) - 1 <= f <= p * (1 + 2.0 ** -45) + 1, i


def test_rotary_of_neither_side(gdn):  # noqa: F811
    i, w = torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(TypeError, match="k must be"):
        gdn.gdn_rotary(None, None, i, w)
    with pytest.raises(TypeError, match="k must be"):
        gdn.gdn_rotary(None, torch.zeros(1, 2, 64), i, w)
    with pytest.raises(ValueError):  # (not on the device)
        gdn.gdn_rotary(None, torch.zeros(1, 2, 64, dtype=torch.bfloat16), i, w)
