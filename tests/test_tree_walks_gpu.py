"""gdn_tree_decode: its two walks give the same bits."""
import pytest
import torch

from tests import tree_util as tu

pytestmark = pytest.mark.gpu

HEADS = [(2, 4, 128), (4, 4, 64)]


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def check(gdn, c, **kw):
    o, st = tu.run_delta(gdn, c, **kw)
    assert st == 0
    tu.assert_close(o, *tu.delta_reference(c))
    return o


@pytest.mark.parametrize("h_k,h_v,d", HEADS)
@pytest.mark.parametrize("m,bounds", [(16, (16, 32, 64)), (32, (32, 64)), (64, (64,)), (29, (32, 64))])
def test_both_walks_give_the_same_bits(gdn, h_k, h_v, d, m, bounds):
    # paths of up to 8 nodes are walked one way, warps that have a longer one another way: a chain of 8, and nodes on it,
    # without and with a ninth level in every 8 nodes behind the chain (a warp takes 8, 16 or 32 nodes)
    short = list(range(-1, 7)) + [u % 7 for u in range(8, m)]
    deep = [u for u in range(8, m) if u % 8 == 7 or u == m - 1]
    long = [7 if u in deep else p for u, p in enumerate(short)]
    assert max(len(tu.path_of(short, u)) for u in range(m)) == 8
    assert {len(tu.path_of(long, u)) for u in deep} == {9}
    same = torch.tensor([u not in deep for u in range(m)], device="cuda")
    outs = []
    for tree in (short, long):
        c = tu.make_delta([tree], h_k, h_v, d, seed=m)
        outs += [check(gdn, c, max_nodes=b) for b in bounds]
    assert all(torch.equal(o[same], outs[0][same]) for o in outs)
