"""gdn_tree_decode: a path under other numbers."""
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
@pytest.mark.parametrize("L,step", [(16, 2), (8, 8), (21, 3), (5, 13)])
def test_a_path_under_other_numbers(gdn, h_k, h_v, d, L, step):
    # the same nodes numbered 0 to L - 1, and every `step`-th, others between them: sums are taken in the order of the
    # numbers, in steps of 16, so the outputs agree to their tolerances (and on the contents of the others to the bit)
    chain = tu.make_delta([list(range(-1, L - 1))], h_k, h_v, d, seed=L)
    want = check(gdn, chain)
    m = (L - 1) * step + 1
    par = [u - step if u % step == 0 else max(-1, u - step - 1) for u in range(m)]
    par = [max(p, -1) for p in par]
    wide = tu.make_delta([par], h_k, h_v, d, seed=L + 100)
    for x in ("q", "k", "v", "g", "beta"):
        wide[x][::step] = chain[x]
    wide["state"][int(wide["slot"][0])] = chain["state"][int(chain["slot"][0])]
    got = check(gdn, wide)
    _, tol = tu.delta_reference(chain)
    tu.assert_close(got[::step], want.double(), 2 * tol)
    for x in ("q", "k", "v", "beta"):
        others = torch.ones(m, dtype=torch.bool, device="cuda")
        others[::step] = False
        wide[x][others] = 0.0625
    again = check(gdn, wide)
    assert torch.equal(again[::step], got[::step])
