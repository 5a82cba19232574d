"""The tree attention's bounded waits, as those of the paged attention: waits that end after one clock cycle are reported,
and the context stays usable."""
import pytest
import torch

from tests import paged_util as pu
from tests import tree_util as tu
from tests.test_paged_timeout_gpu import gdn, short_wait_lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 256), (8, 2, 128), (4, 4, 64)])
def test_timeout_is_reported_and_the_context_survives(gdn, short_wait_lib, h_q, h_kv, d):  # noqa: F811
    lens = [(3000, 1), (700, 64), (129, 4), (2000, 30)]
    c = pu.make_case(lens, h_q, h_kv, d, page=16, seed=31)
    masks = tu.words_of([tu.parents_of(m, "mixed", seed=i) for i, (_, m) in enumerate(lens)])
    saved = gdn._lib
    try:
        gdn._lib = short_wait_lib
        for _ in range(3):
            _, word = tu.run_tree_attention(gdn, c, masks)
            assert word & gdn.GDN_DEV_TIMEOUT, f"no timeout reported (status {word:#x})"
            assert gdn.gdn_status_from_device(word) == gdn.GDN_ERR_TIMEOUT
    finally:
        gdn._lib = saved
    o, word = tu.run_tree_attention(gdn, c, masks)
    assert word == 0
    pu.assert_close(o, *tu.attention_reference(c, masks))
