"""gdn_tree_maps: each node's word and position, bad parents and ranges, padding, capture."""
import pytest
import torch

from tests import tree_util as tu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def call(gdn, parents, cu, kv, stream=None):
    T = parents.numel()
    masks = torch.full((T,), -7, dtype=torch.int64, device="cuda")
    pos = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_tree_maps(parents, cu, kv, masks, pos, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    return masks, pos, int(st.item())


def flat(trees, pad=0):
    return tu.i32(sum((list(p) for p in trees), []) + [-1] * pad)


@pytest.mark.parametrize("sizes", [[1], [2], [31], [32], [33], [63], [64], [1] * 200, [0, 64, 0, 1, 17, 0], list(range(65))])
@pytest.mark.parametrize("shape", tu.SHAPES)
def test_words_and_positions(gdn, sizes, shape):
    trees = [tu.parents_of(m, shape, seed=i) for i, m in enumerate(sizes)]
    ctx = [37 * i % 5000 for i in range(len(sizes))]
    cu = tu.i32(tu.offsets(sizes))
    masks, pos, st = call(gdn, flat(trees, 5), cu, tu.i32([c + m for c, m in zip(ctx, sizes)]))
    want = [c + len(tu.path_of(p, u)) - 1 for c, p in zip(ctx, trees) for u in range(len(p))]
    assert st == 0 and pos.tolist() == want + [0] * 5
    assert torch.equal(masks[:-5], tu.words_of(trees)) and masks[-5:].tolist() == [0] * 5


def test_many_requests(gdn):
    sizes = [(i * 7) % 65 for i in range(6000)]  # more than a wave of blocks
    trees = [tu.parents_of(m, "mixed", seed=i % 50) for i, m in enumerate(sizes)]
    masks, pos, st = call(gdn, flat(trees), tu.i32(tu.offsets(sizes)), tu.i32([m + 3 for m in sizes]))
    assert st == 0 and torch.equal(masks, tu.words_of(trees))
    assert pos.tolist() == [2 + len(tu.path_of(p, u)) for p in trees for u in range(len(p))]


def test_a_parent_that_is_not_before_its_node_is_a_root(gdn):
    par = [-1, 0, 2, 5, -2, 3, 2 ** 31 - 1]
    masks, pos, st = call(gdn, tu.i32(par), tu.i32([0, 7]), tu.i32([17]))
    assert st == gdn.GDN_DEV_BAD_PARENT
    sound = [-1, 0, -1, -1, -1, 3, -1]
    assert torch.equal(masks, tu.words_of([sound]))
    assert pos.tolist() == [10, 11, 10, 10, 10, 11, 10]


def test_bad_lengths(gdn):
    # 65 nodes: zeros; fewer keys than nodes: positions of zero; the request between them is served
    sizes = [65, 3, 4]
    trees = [tu.parents_of(m, "chain") for m in sizes]
    masks, pos, st = call(gdn, flat(trees), tu.i32(tu.offsets(sizes)), tu.i32([100, 2, 14]))
    assert st == gdn.GDN_DEV_BAD_LENGTH
    assert masks.tolist() == [0] * 65 + [1, 3, 7] + [1, 3, 7, 15]
    assert pos.tolist() == [0] * 68 + [10, 11, 12, 13]


def test_ranges_that_run_backwards_or_out_are_skipped(gdn):
    par = flat([[-1, 0, 1, 2]] * 2, pad=2)
    # the middle request's range runs backwards; the last one's begins a token early, whose parent (2) is not before it
    masks, pos, st = call(gdn, par, tu.i32([0, 4, 3, 8]), tu.i32([4, 4, 5]))
    assert st == gdn.GDN_DEV_BAD_LENGTH | gdn.GDN_DEV_BAD_PARENT and masks[:3].tolist() == [1, 3, 7] and masks[8:].tolist() == [0, 0]
    masks, pos, st = call(gdn, par, tu.i32([-2, 4, 8, 99]), tu.i32([4, 4, 4]))
    assert st == gdn.GDN_DEV_BAD_LENGTH and masks[4:8].tolist() == [1, 3, 7, 15] and masks[8:].tolist() == [-7, -7]


def test_no_requests_and_no_tokens(gdn):
    masks, pos, st = call(gdn, tu.i32([0, 0, 0]), tu.i32([0]), tu.i32([]))
    assert st == 0 and masks.tolist() == [0] * 3 and pos.tolist() == [0] * 3
    call(gdn, tu.i32([]), tu.i32([0, 0]), tu.i32([5]))


def test_replays_for_other_trees(gdn):
    a, b = ([tu.parents_of(m, s, 3) for m in (20, 40)] for s in ("mixed", "forest"))
    parents, cu, kv = flat(a), tu.i32([0, 20, 60]), tu.i32([120, 50])
    masks = torch.zeros(60, dtype=torch.int64, device="cuda")
    pos = torch.zeros(60, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    gdn.gdn_tree_maps(parents, cu, kv, masks, pos, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_tree_maps(parents, cu, kv, masks, pos)
    parents.copy_(flat(b))
    kv.copy_(tu.i32([99, 1000]))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(masks, tu.words_of(b))
    assert pos.tolist() == [c + len(tu.path_of(p, u)) - 1 for c, p in zip((79, 960), b) for u in range(len(p))]
