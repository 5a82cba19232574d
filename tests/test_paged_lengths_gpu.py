"""Token ranges and lengths of a step that leave little or nothing to attend, or make no sense."""
import pytest
import torch

from tests import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def test_a_captured_step_of_no_tokens_between_others(gdn):
    # More items than blocks by the bound, so that they are counted out, and contexts too short to be split: nothing but the
    # attention stands between the counter's reset and what follows.  All its lengths are zero in every other replay.
    n = 400
    c = pu.make_case([(1 + 7 * i % 250, 1) for i in range(n)], 4, 2, 64, page=16, seed=72)
    want, st = pu.run_attention(gdn, c, max_kv_len=256)
    assert st == 0
    cu, kv = c["cu"].clone(), c["kv"].clone()
    ws = torch.full((gdn.gdn_paged_attention_workspace_bytes(4, 2, 64, n, n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    o, word = torch.empty_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_paged_attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], o, max_kv_len=256, workspace=ws,
                                dev_status=word)
    for _ in range(30):
        c["cu"].zero_()
        c["kv"].zero_()
        o.fill_(float("nan"))
        graph.replay()
        none = o.clone()
        c["cu"].copy_(cu)
        c["kv"].copy_(kv)
        o.fill_(float("nan"))
        graph.replay()
        assert not none.any() and torch.equal(o, want)
    assert word.item() == 0
