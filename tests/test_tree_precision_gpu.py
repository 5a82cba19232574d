"""gdn_tree_decode: how near the nodes' products are, on values that cancel."""
import pytest
import torch

from tests import tree_util as tu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,max_nodes", [(2, 2), (2, 64), (8, 8), (9, 16), (16, 16), (20, 32), (32, 64), (64, 64)])
def test_products_of_the_nodes(gdn, m, max_nodes, d):
    """A chain whose last node's output is b (1 + y) - y - v0 with b = beta of the last node, 1 + y its value less the
    state's, -1 the first node's factor and v0 its value; the nodes between have beta 0.

    Every number but b and 1 + y is held exactly in 8 bits (y, v0, the factors of 1 and -1), the sums are exact but for fp32's
    roundings.  So b (1 + y) is all that the splits take something of: each factor is the sum of two bf16, the upper one off
    by 2^-8 of it at most, the rest of that by 2^-17 of the factor (half a step of a number up to 2^-8), and the product of
    the two rests is left out: 2^-16 + 2 * 2^-17 = 2^-15 of it.  v0 takes nearly all of it away."""
    h = 16
    gen = torch.Generator().manual_seed(m + d)
    b = 1 + torch.rand(h, generator=gen)                                   # any 24 bits
    b[:4] = torch.tensor([1 + 2.0 ** -7 - 2.0 ** -15, 1 + 2.0 ** -7 - 2.0 ** -23, 1 + 2.0 ** -8 - 2.0 ** -16, 1 + 3 * 2.0 ** -8])
    y = torch.rand(d, generator=gen).bfloat16().float() * 2.0 ** -7        # 8 bits
    y[:4] = torch.tensor([2.0 ** -7 - 2.0 ** -15, 2.0 ** -8 - 2.0 ** -16, 2.0 ** -8 + 2.0 ** -15, 2.0 ** -7 - 2.0 ** -14])
    product = b.double()[:, None] * (1 + y.double())
    v0 = (product - y.double()).bfloat16()
    c = tu.make_delta([list(range(-1, m - 1))], 1, h, d, extra_slots=0)
    for name in ("q", "k", "v", "g", "beta", "state"):
        c[name].zero_()
    c["k"][0, 0, 0] = c["k"][-1, 0, 1] = c["q"][-1, 0, 1] = 1.0
    c["k"][1:-1, 0, 2] = 1.0
    c["q"][-1, 0, 0] = -1.0
    c["v"][0], c["v"][-1] = v0.cuda(), 1.0
    c["beta"][0], c["beta"][-1] = 1.0, b.cuda()
    c["state"][0, :, :, 1] = -y.cuda()
    o, st = tu.run_delta(gdn, c, max_nodes=max_nodes)
    want = product - y.double() - v0.double()
    tol = 2.0 ** -15 * product + 2.0 ** -8 * want.abs() + 8 * 2.0 ** -24 * 4  # the output's half step; eight sums under 4
    err = (o[-1].double().cpu() - want).abs()
    assert st == 0 and (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"


@pytest.mark.parametrize("m", [4, 12, 40])
def test_the_largest_finite_values(gdn, m):
    # shares between bf16's largest number and fp32's: small factors make finite outputs of them, and others see nothing
    h, d = 2, 128
    c = tu.make_delta([[-1] + [u - 1 for u in range(1, m - 1)] + [-1]], h, h, d, seed=m, extra_slots=0)
    c["v"].zero_(), c["state"].zero_(), c["k"].zero_(), c["q"].zero_(), c["g"].zero_()
    c["k"][:, :, 0] = c["q"][:, :, 0] = 1.0
    c["beta"][:] = 2.0 ** -60
    c["v"][0, :, 3], c["state"][0, :, 3, 0] = torch.finfo(torch.bfloat16).max, -2.0 ** 119
    o, st = tu.run_delta(gdn, c)
    ref, tol = tu.delta_reference(c)
    assert st == 0 and torch.isfinite(o[0]).all() and torch.isfinite(o[-1]).all()
    tu.assert_close(o, ref, tol)
