"""Host-side refusals of the calls over trees and of the rotary calls, before any CUDA call; the frequencies."""
import ctypes
import math
import os
import shutil
from fractions import Fraction

import pytest
import torch

from tests.test_paged_cpu import BAD_CACHES, FAKE, INVALID, ODD, UNSUPPORTED, WORKSPACE, cache


@pytest.fixture(scope="module")
def gdn():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from linear_attention_serving_gdn_gb300 import _build
    _build.build()
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def maps(gdn, n=2, T=4, parents=FAKE, cu=FAKE, kv=FAKE, masks=FAKE, pos=FAKE):
    return gdn.load_library().gdn_tree_maps(n, T, parents, cu, kv, masks, pos, None, None)


def attention(gdn, c=None, n=2, T=4, h_q=4, scale=1.0, max_kv=0, q=FAKE, q_stride=512, table=FAKE, width=4, stride=4,
              cu=FAKE, kv=FAKE, masks=FAKE, o=FAKE, ws=None, ws_bytes=0):
    c = cache(gdn) if c is None else c
    return gdn.load_library().gdn_tree_attention(ctypes.byref(c), n, T, h_q, scale, max_kv, q, q_stride, table, width,
                                                 stride, cu, kv, masks, o, ws, ws_bytes, None, None)


def decode(gdn, dims=(4, 8, 128, 128, 1.0), n=2, most=8, T=4, cu=FAKE, masks=FAKE, q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE,
           state=FAKE, slots=4, src=FAKE, o=FAKE):
    d = gdn.Dims(*dims)
    return gdn.load_library().gdn_tree_decode(ctypes.byref(d), n, most, T, cu, masks, q, k, v, g, beta, state, slots, src,
                                              o, None, None)


def side(gdn, x=0x10000, out=0x20000, heads=4, xt=512, xh=128, ot=512, oh=128):
    return gdn.RotarySide(x, out, heads, xt, xh, ot, oh)


def rotary(gdn, dtype=0, T=4, d=128, rot=64, magnitude=1.0, pos=FAKE, freq=FAKE, q=None, k=None, **fields):
    q = side(gdn, **fields) if q is None else q
    return gdn.load_library().gdn_rotary(dtype, T, d, rot, 0, magnitude, pos, freq, ctypes.byref(q) if q else None,
                                         ctypes.byref(k) if k else None, None)


@pytest.mark.parametrize("args,status", [
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(parents=None), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(masks=None), INVALID), (dict(pos=None), INVALID)])
def test_bad_maps_arguments(gdn, args, status):
    assert maps(gdn, **args) == status
    assert maps(gdn, T=0, parents=None) == 0


@pytest.mark.parametrize("fields,status", BAD_CACHES)
def test_bad_caches(gdn, fields, status):
    assert attention(gdn, cache(gdn, **fields)) == status


@pytest.mark.parametrize("args,status", [
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(h_q=0), INVALID), (dict(h_q=5), INVALID),
    (dict(h_q=512), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(max_kv=-1), INVALID), (dict(max_kv=65), INVALID), (dict(q=None), INVALID),
    (dict(q=ODD), INVALID), (dict(q_stride=504), INVALID), (dict(table=None), INVALID), (dict(stride=3), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(masks=None), INVALID), (dict(o=None), INVALID),
    (dict(ws=ctypes.c_void_p(0x10010)), WORKSPACE)])
def test_bad_attention_arguments(gdn, args, status):
    assert attention(gdn, **args) == status
    assert attention(gdn, T=0, masks=None, q=None, o=None) == 0


@pytest.mark.parametrize("args,status", [
    (dict(dims=(4, 8, 96, 96, 1.0)), UNSUPPORTED), (dict(dims=(4, 8, 128, 64, 1.0)), UNSUPPORTED),
    (dict(dims=(4, 6, 128, 128, 1.0)), INVALID), (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(most=0), INVALID),
    (dict(most=65), INVALID), (dict(slots=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(n=1 << 29), UNSUPPORTED),
    (dict(cu=None), INVALID), (dict(masks=None), INVALID), (dict(q=None), INVALID), (dict(k=ODD), INVALID),
    (dict(v=None), INVALID), (dict(g=None), INVALID), (dict(beta=None), INVALID), (dict(state=ODD), INVALID),
    (dict(state=ctypes.c_void_p(0x10010)), INVALID), (dict(src=None), INVALID), (dict(o=ODD), INVALID)])
def test_bad_decode_arguments(gdn, args, status):
    assert decode(gdn, **args) == status
    assert decode(gdn, T=0) == 0 and decode(gdn, n=0) == 0


@pytest.mark.parametrize("args,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(d=0), INVALID),
    (dict(d=1032), UNSUPPORTED), (dict(rot=0), INVALID), (dict(rot=63), INVALID), (dict(rot=130), INVALID),
    (dict(magnitude=float("inf")), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID), (dict(x=None), INVALID),
    (dict(out=None), INVALID), (dict(x=0x10001), INVALID), (dict(heads=-1), INVALID), (dict(heads=1 << 17), UNSUPPORTED),
    (dict(xt=-8), INVALID), (dict(xh=-8), INVALID), (dict(oh=64), INVALID), (dict(ot=0), INVALID),
    (dict(out=0x10000, ot=1024), INVALID)])
def test_bad_rotary_arguments(gdn, args, status):
    assert rotary(gdn, **args) == status


def test_rotary_of_nothing(gdn):
    assert rotary(gdn, T=0) == 0
    assert rotary(gdn, heads=0, x=None, out=None) == 0
    assert gdn.load_library().gdn_rotary(0, 4, 128, 64, 0, 1.0, FAKE, FAKE, None, None, None) == INVALID


SCALINGS = [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0), ("yarn", 16.0, 4096), ("yarn", 40.0, 32768)]


@pytest.mark.parametrize("rot", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 1000000.0])
@pytest.mark.parametrize("scaling,factor,length", SCALINGS)
def test_frequencies(gdn, rot, base, scaling, factor, length):
    if scaling == "ntk" and rot == 2:
        with pytest.raises(gdn.GdnError):
            gdn.gdn_rotary_frequencies(rot, base, scaling, factor)
        return
    got = gdn.gdn_rotary_frequencies(rot, base, scaling, factor, original_length=length).tolist()
    b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
    want = [b ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        want = [f / factor for f in want]
    if scaling == "yarn":
        at = [rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        want = [f * (1 - r) + f / factor * r for f, r in zip(want, ramp)]
    two_pi = Fraction(884279719003555, 140737488355328) + Fraction(2449293598294706, 10 ** 31)  # its double, and the rest
    for f, w in zip(got, want):
        # powers and logarithms of doubles on both sides: a few parts in 2^53 each; and half a unit of 2^-64
        assert abs(Fraction(f, 1 << 64) * two_pi - Fraction(w)) <= Fraction(w) * Fraction(64, 1 << 53) + Fraction(8, 1 << 64)


@pytest.mark.parametrize("args", [
    (0, 1e4, "none", 1.0), (3, 1e4, "none", 1.0), (64, 1.0, "none", 1.0), (64, float("nan"), "none", 1.0),
    (64, 1e4, "linear", 0.5), (64, 1e4, "ntk", float("inf")), (64, 1e4, "yarn", 4.0, 0), (64, 1e4, "yarn", 4.0, 4096, 1.0, 2.0),
    (64, 1e4, "yarn", 4.0, 4096, 32.0, 0.0)])
def test_bad_frequencies(gdn, args):
    with pytest.raises(gdn.GdnError):
        gdn.gdn_rotary_frequencies(*args)
    with pytest.raises(ValueError):
        gdn.gdn_rotary_frequencies(64, 1e4, "cubic")


def test_binding_checks_its_tensors(gdn):
    # CPU tensors and wrong types never reach the library
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    kc = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16)
    i, w = torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        gdn.gdn_tree_maps(i, i, i, w, i)
    with pytest.raises(ValueError):
        gdn.gdn_tree_attention(q, kc, kc, i[None], i, i, w, q)
    with pytest.raises(ValueError):
        gdn.gdn_tree_decode(q, q, q, w, w, kc, i, i, w, q)
    with pytest.raises(ValueError):
        gdn.gdn_rotary(q, q, i, w)
    with pytest.raises(TypeError):
        gdn.gdn_rotary(q.float(), None, i, w)
