"""Host-side refusals of the paged-cache calls: every bad argument is turned down before any CUDA call."""
import ctypes
import os
import shutil

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def gdn():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from linear_attention_serving_gdn_gb300 import _build
    _build.build()
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def cache(gdn, **kw):
    f = dict(k=0x10000, v=0x10000, dtype=0, page_size=16, h_kv=2, d=128, num_pages=8, k_page_stride=16 * 256,
             k_slot_stride=256, k_head_stride=128, v_page_stride=16 * 256, v_slot_stride=256, v_head_stride=128)
    f.update(kw)
    return gdn.PagedCache(*(f[n] for n, _ in gdn.PagedCache._fields_))


BAD_CACHES = [
    (dict(d=96), UNSUPPORTED), (dict(d=0), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(page_size=0), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(h_kv=0), INVALID), (dict(num_pages=-1), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages=1 << 27), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=0x10008), INVALID),
    (dict(k_slot_stride=260), INVALID), (dict(v_page_stride=0), INVALID), (dict(k_head_stride=-128), INVALID),
    (dict(v_page_stride=1 << 60), INVALID),
]


def attention(gdn, c=None, n=2, T=4, h_q=4, scale=1.0, window=0, max_kv=0, q=FAKE, q_stride=512, table=FAKE, width=4,
              stride=4, cu=FAKE, kv=FAKE, o=FAKE, ws=None, ws_bytes=0):
    c = cache(gdn) if c is None else c
    return gdn.load_library().gdn_paged_attention(ctypes.byref(c), n, T, h_q, scale, window, max_kv, q, q_stride, table,
                                                  width, stride, cu, kv, o, ws, ws_bytes, None, None)


def write(gdn, c=None, T=4, k=FAKE, ks=256, kh=128, v=FAKE, vs=256, vh=128, slots=FAKE):
    c = cache(gdn) if c is None else c
    return gdn.load_library().gdn_paged_kv_write(ctypes.byref(c), T, k, ks, kh, v, vs, vh, slots, None, None)


def maps(gdn, n=2, page=16, pages=8, ctx=FAKE, new=FAKE, table=FAKE, width=4, stride=4, free=FAKE, num_free=3, head=FAKE,
         head_out=FAKE, cu=FAKE, kv=FAKE, cap=4, slots=FAKE, pos=FAKE):
    return gdn.load_library().gdn_paged_maps(n, page, pages, ctx, new, table, width, stride, free, num_free, head,
                                             head_out, cu, kv, cap, slots, pos, None, None)


@pytest.mark.parametrize("fields,status", BAD_CACHES)
def test_bad_caches(gdn, fields, status):
    assert attention(gdn, cache(gdn, **fields)) == status
    assert write(gdn, cache(gdn, **fields)) == status


@pytest.mark.parametrize("args,status", [
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(h_q=0), INVALID), (dict(h_q=5), INVALID),
    (dict(h_q=512), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(T=1 << 30, h_q=4), UNSUPPORTED),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(window=-1), INVALID), (dict(max_kv=-1), INVALID), (dict(max_kv=65), INVALID), (dict(q=None), INVALID),
    (dict(q=ODD), INVALID), (dict(q_stride=504), INVALID), (dict(q_stride=516), INVALID), (dict(table=None), INVALID),
    (dict(width=-1), INVALID), (dict(stride=3), INVALID), (dict(cu=None), INVALID), (dict(kv=None), INVALID),
    (dict(o=None), INVALID), (dict(o=ODD), INVALID), (dict(ws=ctypes.c_void_p(0x10010)), WORKSPACE)])
def test_bad_attention_arguments(gdn, args, status):
    assert attention(gdn, **args) == status


def test_attention_of_no_tokens_does_nothing(gdn):
    assert attention(gdn, T=0, q=None, o=None) == 0
    assert gdn.load_library().gdn_paged_attention(None, 1, 1, 4, 1.0, 0, 0, FAKE, 512, FAKE, 4, 4, FAKE, FAKE, FAKE, None,
                                                  0, None, None) == INVALID


@pytest.mark.parametrize("args,status", [
    (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k=ODD), INVALID), (dict(slots=None), INVALID), (dict(ks=250), INVALID), (dict(vs=0), INVALID),
    (dict(kh=4), INVALID), (dict(vh=-8), INVALID)])
def test_bad_write_arguments(gdn, args, status):
    assert write(gdn, **args) == status
    assert write(gdn, T=0) == 0


@pytest.mark.parametrize("args,status", [
    (dict(n=-1), INVALID), (dict(page=0), INVALID), (dict(pages=-1), INVALID), (dict(pages=1 << 28), UNSUPPORTED),
    (dict(ctx=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID), (dict(width=-1), INVALID),
    (dict(stride=3), INVALID), (dict(num_free=-1), INVALID), (dict(head=None), INVALID), (dict(head_out=None), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(cap=-1), INVALID), (dict(cap=1 << 31), UNSUPPORTED),
    (dict(slots=None), INVALID), (dict(pos=None), INVALID)])
def test_bad_maps_arguments(gdn, args, status):
    assert maps(gdn, **args) == status


def test_workspace_size(gdn):
    size = gdn.gdn_paged_attention_workspace_bytes
    for bad in [(0, 1, 64, 1, 1, 1), (3, 2, 64, 1, 1, 1), (256, 1, 64, 1, 1, 1), (4, 2, 96, 1, 1, 1),
                (4, 2, 64, -1, 1, 1), (4, 2, 64, 1, -1, 1), (4, 2, 64, 1, 1, -1), (4, 2, 64, 1, 1, 1 << 31)]:
        with pytest.raises(ValueError):
            size(*bad)
    assert size(4, 2, 64, 1, 1, 16) >= 0
    # more tokens or longer contexts never need less
    assert size(16, 2, 256, 8, 8, 4096) <= size(16, 2, 256, 8, 9, 4096) <= size(16, 2, 256, 8, 9, 100000)


def test_binding_checks_its_tensors(gdn):
    # CPU tensors and wrong types never reach the library
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    kc = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_paged_attention(q, kc, kc, i[None], i, i, q)
    with pytest.raises(TypeError):
        gdn.gdn_paged_attention(q, kc.float(), kc.float(), i[None], i, i, q)
    with pytest.raises(ValueError):
        gdn.gdn_paged_kv_write(q, q, kc, kc, i)
    with pytest.raises(ValueError):
        gdn.gdn_paged_maps(i, i, i[None], 16, 2, i, i, i, i)
