"""The paged attention's workspace query beside the call's own check of the size, both on the host."""
import itertools

import pytest

from tests.test_paged_cpu import FAKE, WORKSPACE, attention, cache, gdn  # noqa: F401


@pytest.mark.parametrize("h_q,h_kv,d", [(16, 2, 256), (8, 8, 128), (5, 1, 128), (3, 3, 64), (128, 1, 64)])
def test_no_bound_is_enough_for_any_table(gdn, h_q, h_kv, d):  # noqa: F811
    size = gdn.gdn_paged_attention_workspace_bytes
    for n, tokens in itertools.product((1, 7, 300), (1, 5, 129, 5000)):
        any_table = size(h_q, h_kv, d, n, tokens, 0)
        assert all(size(h_q, h_kv, d, n, tokens, kv) <= any_table for kv in (1, 256, 257, 5000, 1 << 17, 1 << 24, 1 << 30))


@pytest.mark.parametrize("width", [17, 64, 4096])
def test_a_call_without_a_bound_wants_no_more_than_the_query(gdn, width):  # noqa: F811
    # one byte less than the table's own bound asks for is refused; no bound in the query covers that
    c = dict(n=2, T=4, h_q=4, width=width, stride=width, max_kv=0, ws=FAKE)
    own = gdn.gdn_paged_attention_workspace_bytes(4, 2, 128, 2, 4, width * 16)
    assert own > 0 and attention(gdn, cache(gdn), **c, ws_bytes=own - 1) == WORKSPACE
    assert gdn.gdn_paged_attention_workspace_bytes(4, 2, 128, 2, 4, 0) >= own
