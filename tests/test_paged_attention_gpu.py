"""Attention over the paged cache against its definition in 64 bits, at the sizes, layouts and masks where it can go
wrong, and its bitwise independence of batch, pages and padding."""
import pytest
import torch

from tests import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def check(gdn, c, window=0, scale=None, max_kv_len=0, status=0):
    o, st = pu.run_attention(gdn, c, window, scale, max_kv_len)
    assert st == status
    ref, tol = pu.reference(c, window, scale)
    pu.assert_close(o, ref, tol)
    return o


HEADS = [(16, 2, 256), (8, 4, 256), (8, 2, 128), (5, 1, 128), (4, 4, 128), (6, 2, 64), (16, 1, 64), (3, 3, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("h_q,h_kv,d", HEADS)
def test_single_tokens(gdn, h_q, h_kv, d, dtype):
    lens = [(kv, 1) for kv in (1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000, 3001)]
    check(gdn, pu.make_case(lens, h_q, h_kv, d, dtype, page=16, seed=1))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("h_q,h_kv,d", HEADS)
def test_chunks(gdn, h_q, h_kv, d, dtype):
    lens = [(300, 300), (129, 1), (700, 37), (128, 128), (1, 1), (1153, 200), (64, 3), (0, 0), (500, 129)]
    check(gdn, pu.make_case(lens, h_q, h_kv, d, dtype, page=32, seed=2))


@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
@pytest.mark.parametrize("page", [16, 32, 48, 80, 128, 256, 1088])
def test_pages_and_layouts(gdn, page, layout):
    lens = [(page + 1, 1), (2 * page, 5), (page - 1, page - 1), (3 * page + 7, 130)]
    check(gdn, pu.make_case(lens, 4, 2, 128, "bf16", page=page, layout=layout, seed=3))


@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 1000, 100000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_window(gdn, d, window):
    lens = [(2000, 1), (2000, 4), (600, 300), (90, 90), (1500, 257)]
    check(gdn, pu.make_case(lens, 6, 2, d, "fp16", page=48, seed=4), window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_see_nothing_are_zero(gdn, d):
    # fewer cached tokens than new ones: the first tokens stand before position 0
    lens = [(0, 3), (2, 5), (0, 0), (100, 140), (0, 1), (7, 1)]
    c = pu.make_case(lens, 8, 2, d, page=16, seed=5, pad=9)
    o = check(gdn, c)
    assert not o[:3].any() and not o[3:6].any() and not o[8:48].any() and not o[-9:].any()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), float("-inf")])
def test_cache_rows_that_no_token_sees_may_hold_anything(gdn, d, junk):
    lens = [(37, 1), (129, 1), (1, 1), (300, 4), (1153, 1), (140, 140)]
    window = 100
    c = pu.make_case(lens, 8, 2, d, page=48, seed=6)
    P = c["page"]
    c["k"][c["unused"].long()] = junk
    c["v"][c["unused"].long()] = junk
    for r, (kv, m) in enumerate(lens):
        for j in list(range(kv, pu.ceil(kv, P) * P)) + list(range(0, max(0, kv - m - window + 1))):
            page = int(c["table"][r, j // P])
            c["k"][page, j % P] = junk
            c["v"][page, j % P] = junk
    o = check(gdn, c, window=window)
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("h_q,h_kv,d,dtype", [(16, 2, 256, "bf16"), (8, 2, 128, "fp16"), (6, 2, 64, "bf16"), (3, 3, 64, "fp16"),
                                              (2, 2, 256, "fp16")])
@pytest.mark.parametrize("window", [0, 150])
def test_what_a_token_does_not_see_has_no_part_in_it(gdn, h_q, h_kv, d, dtype, window):
    """NaN and infinities in keys and values of the chunk's later tokens, and, with a window, of earlier ones."""
    lens = [(300, 40), (1700, 9), (129, 129), (2600, 1), (700, 300)]
    c = pu.make_case(lens, h_q, h_kv, d, dtype, page=16, seed=19)
    bad = {0: [(280, "v", float("nan")), (299, "k", float("nan"))], 1: [(1697, "v", float("inf"))],
           2: [(64, "v", float("-inf")), (128, "v", float("nan"))], 4: [(655, "v", float("nan")), (410, "v", float("inf"))]}
    if window:
        bad[0].append((115, "v", float("nan")))  # the first tokens' windows hold it, the last ones' do not
    for r, where in bad.items():
        for j, side, x in where:
            page = c["table"][r, j // 16].long()
            c[side][page, j % 16, :, 3] = x
    o, st = pu.run_attention(gdn, c, window)
    assert st == 0
    t = 0
    for r, (kv, m) in enumerate(lens):
        for u in range(0, m, 1 if m < 50 else 7):
            one = dict(c, q=c["q"][t + u:t + u + 1], table=c["table"][r:r + 1], lens=[(kv - m + u + 1, 1)])
            ref, tol = pu.reference(one, window)
            got = o[t + u].double()
            finite = torch.isfinite(ref[0])
            # a token that sees such a value shows it, the others come out as if it were not there
            assert torch.equal(finite, torch.isfinite(got)), (r, u)
            seen = [x for j, _, x in bad.get(r, []) if j <= kv - m + u and (not window or j > kv - m + u - window)]
            assert bool(finite.all()) == (not seen)
            if not seen:
                pu.assert_close(got, ref[0], tol[0], f"request {r} token {u}")
        t += m


def test_pages_behind_the_window_are_not_looked_at(gdn):
    lens = [(1000, 1), (1000, 3)]
    c = pu.make_case(lens, 4, 2, 128, page=16, seed=7)
    want = check(gdn, c, window=100)
    c["table"][:, :50] = torch.tensor([-7, 1 << 30], device="cuda", dtype=torch.int32).repeat(25)
    got, st = pu.run_attention(gdn, c, window=100)
    assert st == 0 and torch.equal(got, want)


@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_page_reads_as_zeros_and_is_reported(gdn, bad):
    c = pu.make_case([(200, 2), (90, 1)], 4, 2, 64, page=16, seed=8)
    c["table"][0, 3] = bad
    check(gdn, c, status=gdn.GDN_DEV_BAD_SLOT)


def test_bad_lengths_are_skipped_and_reported(gdn):
    c = pu.make_case([(50, 2), (60, 3), (70, 1)], 4, 2, 64, page=16, seed=9)
    ref, tol = pu.reference(c)
    for bad in (-1, 100000):
        c["kv"][1] = bad
        o, st = pu.run_attention(gdn, c)
        assert st == gdn.GDN_DEV_BAD_LENGTH
        assert not o[2:5].any()
        pu.assert_close(o[:2], ref[:2], tol[:2])
        pu.assert_close(o[5:], ref[5:], tol[5:])
    c["kv"][1] = 60
    # a stated bound that a request exceeds
    o, st = pu.run_attention(gdn, c, max_kv_len=65)
    assert st == gdn.GDN_DEV_BAD_LENGTH and not o[5:].any()
    pu.assert_close(o[:5], ref[:5], tol[:5])
    # token ranges that run backwards or past the tokens there are
    c["cu"][:] = torch.tensor([0, 2, 1, 9], dtype=torch.int32)
    o, st = pu.run_attention(gdn, c)
    assert st == gdn.GDN_DEV_BAD_LENGTH
    pu.assert_close(o[:2], ref[:2], tol[:2])


@pytest.mark.parametrize("scale", [0.0, 1.0, 1e-3])
def test_scale(gdn, scale):
    check(gdn, pu.make_case([(300, 40), (77, 1)], 4, 2, 64, page=16, seed=10, q_gain=0.5), scale=scale)


@pytest.mark.parametrize("d", [64, 256])
def test_scores_that_grow_along_the_keys(gdn, d):
    # every tile raises the running maximum by much more than any rescaling threshold, or falls far below it
    c = pu.make_case([(900, 130), (900, 1)], 4, 2, d, "bf16", page=32, seed=11, q_gain=0.05)
    for r in range(2):
        for j in range(900):
            c["k"][c["table"][r, j // 32].long(), j % 32] *= 0.02
            c["k"][c["table"][r, j // 32].long(), j % 32, :, 0] = (j / 10.0) if r == 0 else (90 - j / 10.0)
    c["q"][..., 0] = 4.0
    check(gdn, c)


def test_infinite_scores_follow_the_formula(gdn):
    c = pu.make_case([(200, 1), (200, 1)], 2, 1, 64, "bf16", page=16, seed=12)
    c["q"][..., 0] = 1.0
    page = c["table"][0, 3].long()
    c["k"][page, 5, 0, 0] = float("-inf")  # weight zero
    page1 = c["table"][1, 3].long()
    c["k"][page1, 5, 0, 0] = float("inf")  # inf - inf
    o, _ = pu.run_attention(gdn, c)
    ref, _ = pu.reference(c)
    # a mean of 200 unit normals with a few heavy weights: A <= 2, and half a step each for weights and output
    pu.assert_close(o[:1], ref[:1], torch.full_like(ref[:1], 2.0 ** -6))
    assert torch.isnan(o[1]).all()


def test_outputs_do_not_depend_on_batch_pages_or_padding(gdn):
    lens = [(2500, 1), (4000, 1), (130, 1), (900, 4), (333, 333), (5000, 200)]
    for h_q, h_kv, d in [(16, 2, 256), (8, 8, 64)]:
        c = pu.make_case(lens, h_q, h_kv, d, page=64, seed=13)
        whole, st = pu.run_attention(gdn, c)
        assert st == 0
        t = 0
        for r, (kv, m) in enumerate(lens):
            one = dict(c, q=c["q"][t:t + m], table=c["table"][r:r + 1].clone(), lens=[(kv, m)],
                       cu=torch.tensor([0, m], dtype=torch.int32, device="cuda"), kv=c["kv"][r:r + 1].clone())
            alone, _ = pu.run_attention(gdn, one)
            assert torch.equal(alone, whole[t:t + m]), f"request {r}"
            # the same with a tight bound, other pages, and padded requests and tokens around it
            pad = torch.cat([one["q"], torch.full_like(one["q"], float("nan"))])
            kk, vv = torch.roll(c["k"], 1, 0), torch.roll(c["v"], 1, 0)
            moved = torch.where(one["table"] >= 0, (one["table"] + 1) % c["k"].shape[0], -1)
            padded = dict(one, q=pad, k=kk, v=vv, table=torch.cat([moved, torch.full_like(moved, -1)]),
                          cu=torch.tensor([0, m, m], dtype=torch.int32, device="cuda"),
                          kv=torch.tensor([kv, 0], dtype=torch.int32, device="cuda"), lens=[(kv, m), (0, 0)])
            got, st = pu.run_attention(gdn, padded, max_kv_len=kv)
            assert st == 0 and torch.equal(got[:m], alone) and not got[m:].any()
            t += m


def test_offsets_past_32_bits(gdn):
    # 2^31 elements and more before the pages in use
    d, h, page = 128, 8, 1088
    pages = (1 << 31) // (page * h * d) + 6
    k = torch.empty((pages, page, h, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    gen = torch.Generator(device="cuda").manual_seed(14)
    kv, m = 3 * page + 11, 5
    k[-4:] = torch.randn(k[-4:].shape, generator=gen, device="cuda").bfloat16()
    v[-4:] = torch.randn(v[-4:].shape, generator=gen, device="cuda").bfloat16()
    table = torch.tensor([[pages - 1, pages - 3, pages - 2, pages - 4]], dtype=torch.int32, device="cuda")
    q = torch.randn((m, 2 * h, d), generator=gen, device="cuda").bfloat16()
    c = {"q": q, "k": k, "v": v, "table": table, "lens": [(kv, m)], "page": page,
         "cu": torch.tensor([0, m], dtype=torch.int32, device="cuda"),
         "kv": torch.tensor([kv], dtype=torch.int32, device="cuda")}
    check(gdn, c)


def test_another_stream_and_empty_calls(gdn):
    c = pu.make_case([(500, 1), (90, 30)], 4, 2, 128, page=16, seed=15)
    want, _ = pu.run_attention(gdn, c)
    got, _ = pu.run_attention(gdn, c, stream=torch.cuda.Stream())
    assert torch.equal(got, want)
    # no requests: every token is padding; no tokens: nothing to do
    none = dict(c, lens=[], table=c["table"][:0], cu=c["cu"][:1], kv=c["kv"][:0])
    o, st = pu.run_attention(gdn, none)
    assert st == 0 and not o.any()
    gdn.gdn_paged_attention(c["q"][:0], c["k"], c["v"], c["table"][:0], c["cu"][:1], c["kv"][:0],
                            want[:0].contiguous())


def test_long_contexts(gdn):
    for h_q, h_kv, d, dtype in [(8, 1, 128, "fp16"), (4, 2, 256, "bf16"), (2, 2, 64, "bf16"), (80, 80, 64, "fp16")]:
        check(gdn, pu.make_case([(40000, 1), (70001, 2)], h_q, h_kv, d, dtype, page=16, seed=16))


def test_many_requests(gdn):
    lens = [(1 + 37 * i % 700, 1) for i in range(700)] + [(400, 133), (90, 90)]
    check(gdn, pu.make_case(lens, 4, 1, 64, page=16, seed=17))


@pytest.mark.parametrize("page", [16, 32, 48, 80, 128, 256, 1088])
def test_pages_of_short_heads(gdn, page):
    # heads of 64: one warp loads K and V, stepping through pages that a tile's end cuts
    lens = [(page + 1, 1), (2 * page, 5), (page - 1, page - 1), (3 * page + 7, 130), (5 * page + 300, 2)]
    check(gdn, pu.make_case(lens, 4, 2, 64, "bf16", page=page, layout="joint", seed=18), window=page + 100)


@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_items_of_all_kinds_after_one_another(gdn, d, window):
    # several items per block: one, two and many key tiles, one and two row tiles, split and whole, in mixed order
    new = [1, 130, 5, 1, 64, 33, 1, 300, 65, 2]
    lens = [(37 * i % 900 + new[i % 10], new[i % 10]) for i in range(60)]
    check(gdn, pu.make_case(lens, 16, 8, d, "fp16", page=32, seed=19), window=window)
