"""The paged attention's bounded waits, exercised on the GPU without a fault: a build of the library whose waits end
after one clock cycle reports the timeout, releases what it holds and leaves the context usable."""
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
    return g._configure(ctypes.CDLL(_build.build_variant("waittest", ["GDN_WAIT_CYCLES=1LL"])))


@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 256), (8, 2, 128), (4, 4, 64)])
def test_timeout_is_reported_and_the_context_survives(gdn, short_wait_lib, h_q, h_kv, d):
    c = pu.make_case([(3000, 1), (700, 300), (129, 4), (2000, 1)], h_q, h_kv, d, page=16, seed=31)
    saved = gdn._lib
    try:
        gdn._lib = short_wait_lib
        for _ in range(3):
            _, word = pu.run_attention(gdn, c)
            assert word & gdn.GDN_DEV_TIMEOUT, f"no timeout reported (status {word:#x})"
            assert gdn.gdn_status_from_device(word) == gdn.GDN_ERR_TIMEOUT
    finally:
        gdn._lib = saved
    o, word = pu.run_attention(gdn, c)
    assert word == 0
    ref, tol = pu.reference(c)
    pu.assert_close(o, ref, tol)
