"""Items that take longer than a wait's limit: whoever waits for a whole item's end waits on while its tiles go by."""
import ctypes

import pytest
import torch

from tests import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


@pytest.fixture(scope="module")
def short_wait_lib():
    import linear_attention_serving_gdn_gb300 as g
    from linear_attention_serving_gdn_gb300 import _build
    # 0.2 ms: many times what a tile takes
    return g._configure(ctypes.CDLL(_build.build_variant("shortwait", ["GDN_WAIT_CYCLES=400000LL"])))


@pytest.mark.parametrize("h_q,h_kv,d,m,kv", [(80, 80, 64, 1280, 120000), (80, 80, 128, 1280, 120000), (80, 80, 256, 640, 120000)])
def test_items_longer_than_the_limit(gdn, short_wait_lib, h_q, h_kv, d, m, kv):
    # 400 unsplit items of 900 tiles, a millisecond and more each; the table goes round 512 keys' pages
    gen = torch.Generator(device="cuda").manual_seed(81)
    page = 64
    k, v = (torch.randn((8, page, h_kv, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((m, h_q, d), generator=gen, device="cuda").bfloat16()
    width = pu.ceil(kv, page)
    c = {"q": q, "k": k, "v": v, "page": page, "lens": [(kv, m)],
         "table": (torch.arange(width, dtype=torch.int32, device="cuda") % 8)[None].contiguous(),
         "cu": torch.tensor([0, m], dtype=torch.int32, device="cuda"), "kv": torch.tensor([kv], dtype=torch.int32, device="cuda")}
    want, st = pu.run_attention(gdn, c)
    assert st == 0
    saved = gdn._lib
    try:
        gdn._lib = short_wait_lib
        got, st = pu.run_attention(gdn, c)
    finally:
        gdn._lib = saved
    assert st == 0
    assert torch.equal(got, want)
