"""gdn_tree_decode on chains against gdn_decode_multi, which commits them."""
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
@pytest.mark.parametrize("L", [1, 2, 8, 9, 16, 24])
def test_a_chain_is_what_is_committed(gdn, h_k, h_v, d, L):
    # verified by one call, committed by the other.  Both lie within the tolerance of the definition: gdn_decode_multi's
    # own roundings, 24 of fp32 a step (a lane's 16 products, the lanes' sums, the update), 2^-24 of what is summed each,
    # are for up to 24 steps 2^-14.8 of it, under the 2^-15 + (d + 64) 2^-23 that it has room for.
    n = 5
    c = tu.make_delta([list(range(-1, L - 1))] * n, h_k, h_v, d, seed=20 + L)
    o = check(gdn, c, max_nodes=L)
    state, multi = c["state"].clone(), torch.empty_like(o)
    gdn.gdn_decode_multi(L, c["q"], c["k"], c["v"], c["g"], c["beta"], state, c["slot"], multi)
    torch.cuda.synchronize()
    _, tol = tu.delta_reference(c)
    tu.assert_close(o, multi.double(), 2 * tol + 2.0 ** -8 * multi.double().abs())
    # and the next tree continues what was committed as one that hangs on the chain does
    nodes = 6
    par = tu.parents_of(nodes, "mixed", seed=L)
    both = tu.make_delta([list(range(-1, L - 1)) + [p + L for p in par]] * n, h_k, h_v, d, seed=40 + L)
    after = tu.make_delta([par] * n, h_k, h_v, d)
    after.update(state=state, slot=c["slot"])
    for x in ("q", "k", "v", "g", "beta"):
        whole = both[x].view(n, L + nodes, *both[x].shape[1:])
        whole[:, :L] = c[x].view(n, L, *c[x].shape[1:])
        after[x] = whole[:, L:].reshape(n * nodes, *both[x].shape[1:]).contiguous()
    both.update(state=c["state"], slot=c["slot"])
    a = check(gdn, after)
    b = check(gdn, both).view(n, L + nodes, h_v, d)[:, L:].reshape(a.shape)
    _, tol = tu.delta_reference(both)
    tol = tol.view(n, L + nodes, h_v, d)[:, L:].reshape(a.shape)
    tu.assert_close(a, b.double(), 2 * (tol + tu.delta_reference(after)[1]))
