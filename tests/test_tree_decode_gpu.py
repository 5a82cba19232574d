"""gdn_tree_decode against the recurrence from each node's parent in 64 bits."""
import pytest
import torch

from tests import tree_util as tu

pytestmark = pytest.mark.gpu

HEADS = [(16, 16, 128), (2, 4, 128), (1, 3, 128), (4, 4, 64), (2, 6, 64)]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def trees_of(sizes, shape):
    return [tu.parents_of(m, shape, seed=i) for i, m in enumerate(sizes)]


def check(gdn, c, status=0, **kw):
    before = c["state"].clone()
    o, st = tu.run_delta(gdn, c, **kw)
    assert st == status and torch.equal(c["state"], before)
    ref, tol = tu.delta_reference(c, kw.get("scale", 1.0))
    tu.assert_close(o, ref, tol)
    return o


@pytest.mark.parametrize("shape", tu.SHAPES)
@pytest.mark.parametrize("h_k,h_v,d", HEADS)
def test_trees(gdn, h_k, h_v, d, shape):
    sizes = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 0, 5]
    c = tu.make_delta(trees_of(sizes, shape), h_k, h_v, d, seed=1, pad=4)
    o = check(gdn, c)
    assert not o[-4:].any()


@pytest.mark.parametrize("most", [1, 5, 8, 9, 16, 23, 32, 41, 64])
@pytest.mark.parametrize("h_k,h_v,d", [HEADS[1], HEADS[4]])
def test_bounds_on_the_nodes(gdn, h_k, h_v, d, most):
    sizes = [most, 1, max(1, most // 2), most]
    c = tu.make_delta(trees_of(sizes, "mixed"), h_k, h_v, d, seed=2)
    o = check(gdn, c, max_nodes=most, scale=0.7)
    wide, _ = tu.run_delta(gdn, c, max_nodes=64, scale=0.7)
    assert torch.equal(o, wide)  # not a bit depends on the bound


@pytest.mark.parametrize("h_k,h_v,d", HEADS)
def test_degenerate_gates(gdn, h_k, h_v, d):
    # full and no forgetting, full and no writing, in one node, a level and everywhere
    c = tu.make_delta(trees_of([33, 20, 8, 12], "mixed"), h_k, h_v, d, seed=3)
    c["g"][:10], c["g"][33:53], c["g"][55] = 0.0, -INF, -200.0
    c["g"][3] = -INF
    c["beta"][20:40], c["beta"][45:], c["beta"][2] = 0.0, 1.0, 0.0
    check(gdn, c)


def test_one_token_is_a_decode_step(gdn):
    n, h, d = 9, 8, 128
    c = tu.make_delta([[-1]] * n, h, h, d, seed=4)
    o = check(gdn, c, max_nodes=1)
    state, want = c["state"].clone(), torch.empty_like(o)
    gdn.gdn_decode_packed(c["q"], c["k"], c["v"], c["g"], c["beta"], state, c["slot"], want)
    _, tol = tu.delta_reference(c)
    tu.assert_close(o, want.double(), 2 * tol + 2.0 ** -8 * want.double().abs())


@pytest.mark.parametrize("h_k,h_v,d", [HEADS[1], HEADS[3]])
def test_a_row_does_not_depend_on_the_batch(gdn, h_k, h_v, d):
    sizes = [12, 64, 1, 30]
    c = tu.make_delta(trees_of(sizes, "mixed"), h_k, h_v, d, seed=5, pad=3)
    o, _ = tu.run_delta(gdn, c)
    cu = c["cu"].tolist()
    for r, m in enumerate(sizes):
        at = slice(cu[r], cu[r + 1])
        one = {x: c[x][at].contiguous() for x in ("q", "k", "v", "g", "beta", "masks")}
        one.update(state=c["state"], slot=c["slot"][r:r + 1], cu=tu.i32([0, m]))
        alone, st = tu.run_delta(gdn, one, max_nodes=m)
        assert st == 0 and torch.equal(alone, o[at])


@pytest.mark.parametrize("h_k,h_v,d", HEADS)
def test_a_node_does_not_see_its_siblings(gdn, h_k, h_v, d):
    # not a bit changes by what is not on a node's path; NaN and infinities show below it
    sizes = [40, 64, 9]
    c = tu.make_delta(trees_of(sizes, "mixed"), h_k, h_v, d, seed=6)
    want, _ = tu.run_delta(gdn, c)
    cu = c["cu"].tolist()
    for r, m in enumerate(sizes):
        w = m // 2
        below = torch.tensor([w in tu.path_of(c["trees"][r], u) for u in range(m)], device="cuda")
        assert below.any() and not below.all()
        for name, column, value in (("v", 5, NAN), ("v", 7, INF), ("k", 2, NAN), ("k", 1, INF), ("q", 0, NAN), ("g", 0, NAN),
                                    ("beta", 0, INF), ("v", slice(None), 3.0)):
            keep = c[name][cu[r] + w].clone()
            c[name][cu[r] + w][..., column] = value
            got, st = tu.run_delta(gdn, c)
            c[name][cu[r] + w] = keep
            rows = torch.zeros(len(want), dtype=torch.bool, device="cuda")
            rows[cu[r]:cu[r + 1]] = below
            assert st == 0 and torch.equal(got[~rows], want[~rows]), (r, name, value)
            head, head_k = (0, 0)  # gates: one value head; v: all of them, one column; k: all
            if name == "v" and value != 3.0:
                assert not torch.isfinite(got[rows][..., column]).any()
                other = [i for i in range(d) if i != column]
                assert torch.equal(got[rows][..., other], want[rows][..., other])
            elif name == "k":
                assert not torch.isfinite(got[rows]).any()
            elif name in ("g", "beta"):
                assert not torch.isfinite(got[rows][:, 0]).any() and torch.equal(got[rows][:, 1:], want[rows][:, 1:])
            elif name == "q":
                assert torch.isnan(got[cu[r] + w]).all()


def test_infinite_values_by_the_definition(gdn):
    c = tu.make_delta([[-1, 0, 0, 1, 2]], 2, 2, 64, seed=7)
    c["v"][0, :, 3], c["v"][1, :, 3], c["v"][2, :, 4] = INF, INF, -INF
    o, _ = tu.run_delta(gdn, c)
    ref, _ = tu.delta_reference(c)
    seen = ~torch.isfinite(ref)
    assert torch.equal(~torch.isfinite(o), seen)


def test_a_state_that_is_not_finite_stays_in_its_row(gdn):
    c = tu.make_delta(trees_of([12, 20, 3], "mixed"), 2, 4, 128, seed=8)
    want, _ = tu.run_delta(gdn, c)
    c["state"][int(c["slot"][1]), 2, 77, 5] = NAN
    got, st = tu.run_delta(gdn, c)
    assert st == 0 and torch.isnan(got[12:32, 2, 77]).all()
    got[12:32, 2, 77] = want[12:32, 2, 77]
    assert torch.equal(got, want)


def test_refused_and_padded_rows(gdn):
    sizes = [20, 5, 7, 6, 9]
    c = tu.make_delta(trees_of(sizes, "mixed"), 2, 2, 128, seed=9)
    want, _ = tu.run_delta(gdn, c)
    c["slot"][1], c["slot"][2] = -1, 10 ** 6
    o, st = tu.run_delta(gdn, c, max_nodes=16)
    assert st == gdn.GDN_DEV_BAD_SLOT | gdn.GDN_DEV_BAD_LENGTH
    assert not o[:32].any() and torch.equal(o[32:], want[32:])
    # a range that runs backwards is skipped, and so is one past the last end
    c["slot"][1:3] = 0
    c["cu"][3] = 24
    o, st = tu.run_delta(gdn, c)
    assert st == gdn.GDN_DEV_BAD_LENGTH and torch.equal(o[:20], want[:20]) and torch.equal(o[38:], want[38:])
    c["cu"][3], c["cu"][5] = 32, 37
    o, st = tu.run_delta(gdn, c)
    assert st == gdn.GDN_DEV_BAD_LENGTH and torch.isnan(o[32:37]).all() and not o[37:].any()


def test_nothing_to_do(gdn):
    c = tu.make_delta([[], [], []], 2, 2, 64, seed=10, pad=2)
    o, st = tu.run_delta(gdn, c)
    assert st == 0 and not o.any()
    c = tu.make_delta([], 2, 2, 64, seed=10)
    assert tu.run_delta(gdn, c)[0].shape[0] == 0


def test_replays_for_other_trees(gdn):
    c = tu.make_delta(trees_of([12, 30], "mixed"), 2, 4, 128, seed=11)
    o = torch.empty_like(c["v"])
    args = (c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], c["slot"], c["cu"], c["masks"], o)
    gdn.gdn_tree_decode(*args, max_nodes=32)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_tree_decode(*args, max_nodes=32)
    c["trees"] = trees_of([20, 22], "forest")
    c["masks"].copy_(tu.words_of(c["trees"]))
    c["cu"].copy_(tu.i32([0, 20, 42]))
    g.replay()
    torch.cuda.synchronize()
    tu.assert_close(o, *tu.delta_reference(c))
    other, st = tu.run_delta(gdn, c, stream=torch.cuda.Stream())
    assert st == 0 and torch.equal(other, o)


@pytest.mark.parametrize("h_k,h_v,d", [HEADS[1], HEADS[3]])
def test_a_long_path_beside_short_ones_changes_no_bit(gdn, h_k, h_v, d):
    # short paths and long ones are walked in different ways
    short = tu.parents_of(20, "mixed", seed=3)
    assert max(len(tu.path_of(short, u)) for u in range(20)) <= 16
    both = short + [19] + list(range(20, 50))
    c = tu.make_delta([both], h_k, h_v, d, seed=12)
    o = check(gdn, c)
    c.update(trees=[short], masks=c["masks"][:20].contiguous(), cu=tu.i32([0, 20]))
    c.update({x: c[x][:20].contiguous() for x in ("q", "k", "v", "g", "beta")})
    alone, st = tu.run_delta(gdn, c)
    assert st == 0 and torch.equal(alone, o[:20])


def test_rows_that_share_a_slot(gdn):
    c = tu.make_delta(trees_of([12, 12, 40], "mixed"), 2, 4, 128, seed=13)
    c["slot"][:] = c["slot"][0].clone()
    check(gdn, c)


def test_two_calls_at_once(gdn):
    sizes = [30] * 40
    cs = [tu.make_delta(trees_of(sizes, shape), 4, 8, 128, seed=14 + i) for i, shape in enumerate(("mixed", "forest"))]
    wants = [tu.run_delta(gdn, c)[0] for c in cs]
    outs, streams = [[torch.empty_like(w) for _ in range(8)] for w in wants], [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for i in range(8):
        for c, out, s in zip(cs, outs, streams):
            gdn.gdn_tree_decode(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], c["slot"], c["cu"], c["masks"],
                                out[i], max_nodes=32, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for out, w in zip(outs, wants) for o in out)


def test_states_far_apart(gdn):
    # slots whose offsets pass 2^31 elements and 2^33 bytes
    c = tu.make_delta(trees_of([9, 33], "mixed"), 16, 32, 128, seed=16)
    want, _ = tu.run_delta(gdn, c)
    n = (1 << 31) // (32 * 128 * 128) + 3
    far = torch.empty((n, 32, 128, 128), device="cuda")
    far[0], far[n - 1] = c["state"][int(c["slot"][0])], c["state"][int(c["slot"][1])]
    c.update(state=far, slot=tu.i32([0, n - 1]))
    o, st = tu.run_delta(gdn, c)
    assert st == 0 and torch.equal(o, want)


def test_a_state_off_its_boundary_is_refused(gdn):
    c = tu.make_delta([[-1, 0]], 2, 2, 64, seed=17)
    flat = torch.zeros(c["state"].numel() + 4, device="cuda")
    c["state"] = flat[4:].view(c["state"].shape)
    assert c["state"].data_ptr() % 32 == 16
    with pytest.raises(RuntimeError):
        tu.run_delta(gdn, c)


@pytest.mark.parametrize("h_k,h_v,d", HEADS)
def test_a_node_beside_a_long_path_does_not_show(gdn, h_k, h_v, d):
    # a chain with a leaf at each of its nodes; NaN and infinities in a leaf, and in a node of the chain
    sizes = [14, 32, 64]
    trees = [[max(-1, u - 2 if u % 2 == 0 else u - 1) for u in range(m)] for m in sizes]
    assert max(len(tu.path_of(trees[-1], u)) for u in range(64)) == 33
    c = tu.make_delta(trees, h_k, h_v, d, seed=18)
    want = check(gdn, c)
    cu = c["cu"].tolist()
    for r, m in enumerate(sizes):
        for w in (m // 2 + 1 - m // 2 % 2, m // 2 - m // 2 % 2):  # odd: a leaf; even: on the chain
            below = torch.tensor([w in tu.path_of(trees[r], u) for u in range(m)], device="cuda")
            assert int(below.sum()) == 1 if w % 2 else below.any() and not below.all()
            rows = torch.zeros(len(want), dtype=torch.bool, device="cuda")
            rows[cu[r]:cu[r + 1]] = below
            for name, value in (("k", NAN), ("k", INF), ("v", NAN), ("v", INF), ("q", NAN), ("g", NAN), ("beta", INF)):
                keep = c[name][cu[r] + w].clone()
                c[name][cu[r] + w] = value
                got, st = tu.run_delta(gdn, c)
                c[name][cu[r] + w] = keep
                assert st == 0 and torch.equal(got[~rows], want[~rows]), (r, w, name, value)
                assert not torch.isfinite(got[cu[r] + w]).any()
                if name != "q":
                    assert not torch.isfinite(got[rows]).any()
