"""gdn_tree_attention against its definition in 64 bits."""
import pytest
import torch

from tests import paged_util as pu
from tests import tree_util as tu

pytestmark = pytest.mark.gpu

HEADS = [(16, 2, 256, "bf16"), (2, 2, 256, "fp16"), (8, 2, 128, "fp16"), (5, 1, 128, "bf16"), (6, 2, 64, "bf16"), (3, 3, 64, "fp16"),
         (32, 1, 64, "bf16")]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def case(lens, heads, shape="mixed", **kw):
    h_q, h_kv, d, dtype = heads
    c = pu.make_case(lens, h_q, h_kv, d, dtype, **kw)
    c["trees"] = [tu.parents_of(m, shape, seed=i) for i, (_, m) in enumerate(lens)]
    pad = torch.zeros(c["q"].shape[0] - sum(m for _, m in lens), dtype=torch.int64, device="cuda")
    return c, torch.cat([tu.words_of(c["trees"]), pad])


def check(gdn, c, masks, status=0, **kw):
    o, st = tu.run_tree_attention(gdn, c, masks, **kw)
    assert st == status
    pu.assert_close(o, *tu.attention_reference(c, masks, kw.get("scale")))
    return o


@pytest.mark.parametrize("shape", tu.SHAPES)
@pytest.mark.parametrize("heads", HEADS)
def test_trees(gdn, heads, shape):
    # a single token, trees that start at, end at and lie across a key tile's border, a whole tree without a context
    lens = [(1, 1), (200, 1), (64, 64), (128, 17), (150, 40), (192, 64), (130, 2), (300, 64), (1000, 33)]
    c, masks = case(lens, heads, shape, page=48, seed=1, pad=3)
    o = check(gdn, c, masks)
    assert not o[-3:].any()


@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
@pytest.mark.parametrize("page", [16, 64, 1088])
@pytest.mark.parametrize("heads", [HEADS[0], HEADS[2], HEADS[4]])
def test_layouts(gdn, heads, page, layout):
    c, masks = case([(700, 30), (1200, 64), (90, 5)], heads, page=page, layout=layout, seed=2)
    check(gdn, c, masks, scale=0.03)


@pytest.mark.parametrize("heads", HEADS)
def test_long_contexts_are_split(gdn, heads):
    c, masks = case([(9000, 12), (20000, 64), (5000, 1)], heads, page=64, seed=3)
    check(gdn, c, masks, max_kv_len=20000)


@pytest.mark.parametrize("heads", HEADS)
def test_any_nodes_before(gdn, heads):
    # words that are no tree's: any nodes before, none, and the node itself left out; bits of nodes behind it count for nothing
    lens = [(64, 64), (40, 40), (500, 64), (7, 7)]
    c, masks = case(lens, heads, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(9)
    masks = torch.randint(-2 ** 62, 2 ** 62, masks.shape, generator=gen, device="cuda")
    masks[5], masks[70], masks[110], masks[-7:] = 0, 0, 0, 0
    o = check(gdn, c, masks)
    assert not o[5].any() and not o[70].any() and not o[-7:].any() and o[110].any()


@pytest.mark.parametrize("heads", HEADS)
def test_a_chain_is_causal_attention(gdn, heads):
    lens = [(300, 64), (129, 3), (5000, 20), (1, 1), (64, 64)]
    c, masks = case(lens, heads, "chain", page=32, seed=5)
    o, st = tu.run_tree_attention(gdn, c, masks)
    want, st2 = pu.run_attention(gdn, c)
    assert st == st2 == 0 and torch.equal(o, want)


@pytest.mark.parametrize("heads", [HEADS[0], HEADS[2], HEADS[4]])
def test_a_request_does_not_depend_on_the_batch(gdn, heads):
    lens = [(300, 64), (4000, 20), (1, 1), (700, 40)]
    c, masks = case(lens, heads, page=16, seed=6, pad=2)
    o, _ = tu.run_tree_attention(gdn, c, masks)
    again, _ = tu.run_tree_attention(gdn, c, masks, fill=0.0)
    assert torch.equal(o, again)
    t = 0
    for r, (kv, m) in enumerate(lens):
        one = dict(c, q=c["q"][t:t + m], table=c["table"][r:r + 1], cu=tu.i32([0, m]), kv=c["kv"][r:r + 1], lens=[(kv, m)])
        alone, _ = tu.run_tree_attention(gdn, one, masks[t:t + m].contiguous(), max_kv_len=kv)
        assert torch.equal(alone, o[t:t + m])
        t += m


@pytest.mark.parametrize("heads", HEADS)
def test_a_node_does_not_see_its_siblings(gdn, heads):
    # not a bit changes by what is not on a node's path, NaN and infinities included
    lens = [(200, 40), (129, 64), (1500, 12), (30, 30)]
    c, masks = case(lens, heads, "mixed", page=16, seed=7)
    want, _ = tu.run_tree_attention(gdn, c, masks)
    t = 0
    for r, (kv, m) in enumerate(lens):
        w = m // 2
        j = kv - m + w
        page, row = c["table"][r, j // 16].long(), j % 16
        keep = c["k"][page, row].clone(), c["v"][page, row].clone()
        for k_val, v_val in ((NAN, NAN), (1.0, INF), (-INF, 2.0), (NAN, -INF)):
            c["k"][page, row], c["v"][page, row, :, 3] = k_val, v_val
            got, st = tu.run_tree_attention(gdn, c, masks)
            sees = torch.zeros(len(masks), dtype=torch.bool)
            for u in range(m):
                sees[t + u] = w in tu.path_of(c["trees"][r], u)
            assert st == 0 and sees.any() and not sees[t:t + m].all()
            assert torch.equal(got[~sees], want[~sees]), (r, k_val, v_val)
            if v_val != 2.0:
                assert not torch.isfinite(got[sees][..., 3]).any()
            c["k"][page, row], c["v"][page, row] = keep
        t += m


@pytest.mark.parametrize("heads", [HEADS[0], HEADS[2], HEADS[5]])
def test_values_that_are_not_finite_show_below_them(gdn, heads):
    lens = [(200, 40), (700, 64)]
    c, masks = case(lens, heads, "forest", page=16, seed=8, q_gain=0.5)
    for r, (kv, m) in enumerate(lens):
        for w, val in ((3, INF), (10, -INF), (m - 2, NAN), (20, INF)):
            j = kv - m + w
            c["v"][c["table"][r, j // 16].long(), j % 16, :, w % 7] = val
    o, st = tu.run_tree_attention(gdn, c, masks)
    ref, tol = tu.attention_reference(c, masks)
    assert st == 0 and torch.equal(torch.isnan(o), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert torch.equal(o[inf].double(), ref[inf])
    ok = torch.isfinite(ref)
    pu.assert_close(o[ok], ref[ok], tol[ok])


@pytest.mark.parametrize("heads", [HEADS[0], HEADS[2], HEADS[4]])
def test_refused_requests(gdn, heads):
    # more than 64 nodes, a negative length, a length over the bound: zeros; backwards: skipped; the others are served
    lens = [(300, 65), (200, 20), (500, 4), (90, 90), (100, 6)]
    c, masks = case([(kv, m) for kv, m in lens], heads, seed=9)
    c["kv"][2] = -3
    o, st = tu.run_tree_attention(gdn, c, masks)
    assert st == gdn.GDN_DEV_BAD_LENGTH
    ref, tol = tu.attention_reference(dict(c, lens=[(0, 65), (200, 20), (0, 4), (0, 90), (100, 6)]), masks)
    pu.assert_close(o, ref, tol)
    assert not o[:65].any() and not o[85:179].any()


def test_a_bad_page_reads_as_zeros(gdn):
    c, masks = case([(200, 20), (300, 64)], HEADS[2], page=16, seed=10)
    c["table"][0, 3], c["table"][1, 17] = -5, 10 ** 6
    o, st = tu.run_tree_attention(gdn, c, masks)
    assert st == gdn.GDN_DEV_BAD_SLOT
    pu.assert_close(o, *tu.attention_reference(c, masks))


def test_fewer_keys_than_nodes(gdn):
    # nodes that stand before the first key see the keys of none of theirs
    c, masks = case([(5, 9), (3, 64)], HEADS[0], seed=11)
    o = check(gdn, c, masks)
    assert not o[:4].any()


@pytest.mark.parametrize("heads", [HEADS[0], HEADS[3], HEADS[5]])
def test_replays_for_other_trees(gdn, heads):
    lens = [(2000, 30), (400, 64), (64, 8)]
    c, masks = case(lens, heads, page=16, seed=12)
    T, h_q, d = c["q"].shape
    ws = torch.empty(gdn.gdn_paged_attention_workspace_bytes(h_q, heads[1], d, 3, T, 2048), dtype=torch.uint8, device="cuda")  # (more than the call needs)
    o = torch.empty((T, h_q, d), dtype=c["q"].dtype, device="cuda")
    args = (c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], masks, o)
    gdn.gdn_tree_attention(*args, max_kv_len=2000, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_tree_attention(*args, max_kv_len=2000, workspace=ws)
    c["trees"] = [tu.parents_of(m, "forest", seed=77 + i) for i, (_, m) in enumerate(lens)]
    masks.copy_(tu.words_of(c["trees"]))
    g.replay()
    torch.cuda.synchronize()
    pu.assert_close(o, *tu.attention_reference(c, masks))
    other, st = tu.run_tree_attention(gdn, c, masks, max_kv_len=2000, stream=torch.cuda.Stream())
    assert st == 0 and torch.equal(other, o)


@pytest.mark.parametrize("heads", [HEADS[0], HEADS[2], HEADS[5]])
def test_pages_far_apart(gdn, heads):
    # a cache whose offsets pass 2^31 elements
    c, masks = case([(300, 20), (90, 64)], heads, page=64, seed=20)
    want, _ = tu.run_tree_attention(gdn, c, masks)
    used = c["k"].shape[0]
    n = (1 << 31) // c["k"][0].numel() + used + 1
    for x in "kv":
        far = torch.empty((n,) + tuple(c[x].shape[1:]), dtype=c[x].dtype, device="cuda")
        far[n - used:] = c[x]
        c[x] = far
    c["table"] = torch.where(c["table"] >= 0, c["table"] + (n - used), c["table"])
    o, st = tu.run_tree_attention(gdn, c, masks)
    assert st == 0 and torch.equal(o, want)


@pytest.mark.parametrize("heads", [HEADS[0], HEADS[2]])
def test_two_calls_at_once(gdn, heads):
    cs = [case([(5000, 30), (700, 64), (9000, 3)] * 3, heads, shape, page=64, seed=21 + i) for i, shape in enumerate(("mixed", "flat"))]
    wants = [tu.run_tree_attention(gdn, c, masks)[0] for c, masks in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    jobs = []
    for (c, masks), want in zip(cs, wants):
        T, h_q, d = c["q"].shape
        n = gdn.gdn_paged_attention_workspace_bytes(h_q, c["k"].shape[2], d, len(c["lens"]), T, c["table"].shape[1] * 64)
        jobs.append((torch.empty(n, dtype=torch.uint8, device="cuda"), [torch.empty_like(want) for _ in range(6)]))
    torch.cuda.synchronize()
    for i in range(6):
        for (c, masks), (ws, outs), s in zip(cs, jobs, streams):
            gdn.gdn_tree_attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], masks, outs[i], workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for (_, outs), w in zip(jobs, wants) for o in outs)


def test_requests_that_share_pages(gdn):
    # a common prefix, and one request drafted twice in one call (its own pages read by both)
    c, masks = case([(500, 12), (500, 40)], HEADS[0], page=64, seed=23)
    c["table"][1, :7] = c["table"][0, :7]
    check(gdn, c, masks)


@pytest.mark.parametrize("heads", HEADS)
def test_a_part_of_which_a_node_sees_nothing(gdn, heads):
    # contexts that end where a part of the keys ends, and nodes that see no node: their last part is empty
    lens = [(ctx + m, m) for ctx, m in ((2048, 20), (2048, 64), (1920, 1), (1920, 5), (384, 3), (0, 7))]
    c, masks = case(lens, heads, page=64, seed=24)
    masks[::2] = 0
    want = check(gdn, c, masks)
    # and what they do not see has no part in it
    for r, (kv, m) in enumerate(lens):
        for j in range(kv - m, kv):
            c["k"][c["table"][r, j // 64].long(), j % 64] = NAN
            c["v"][c["table"][r, j // 64].long(), j % 64] = INF
    o, st = tu.run_tree_attention(gdn, c, masks)
    blind = masks == 0
    assert st == 0 and torch.equal(o[blind], want[blind])
