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


def behind_empty(c, n):
    """The case's requests behind n empty ones."""
    return dict(c, lens=[(0, 0)] * n + c["lens"],
                table=torch.cat([torch.full((n, c["table"].shape[1]), -1, dtype=torch.int32, device="cuda"), c["table"]]),
                cu=torch.cat([c["cu"][:1].expand(n), c["cu"]]), kv=torch.cat([torch.zeros_like(c["kv"][:1]).expand(n), c["kv"]]))


@pytest.mark.parametrize("empty", [0, 50000])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("last", [3, 0, -1])
def test_a_range_that_runs_backwards_leaves_the_others_whole(gdn, d, last, empty):
    # The last request ends before it begins, inside or before the tokens of the one before it.  (Behind many empty ones the
    # padding's zeros are written long after that one's result.)
    c = pu.make_case([(150, 5), (60, 1)], 4, 2, d, page=16, seed=71, pad=3)
    ref, tol = pu.reference(dict(c, lens=[(150, 5)]))
    c["cu"][:] = torch.tensor([0, 5, last], dtype=torch.int32)
    c = behind_empty(c, empty)
    for _ in range(3):
        o, st = pu.run_attention(gdn, c)
        assert st == gdn.GDN_DEV_BAD_LENGTH
        pu.assert_close(o[:5], ref[:5], tol[:5])
        assert not o[5:].any()


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
