"""NaN and infinities in what a token sees show in its output as the definition has them; in what it does not see they
have no part in it."""
import pytest
import torch

from tests import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


HEADS = [(16, 2, 256, "bf16"), (2, 2, 256, "fp16"), (8, 2, 128, "fp16"), (5, 1, 128, "bf16"), (6, 2, 64, "bf16"), (3, 3, 64, "fp16")]
NAN, INF = float("nan"), float("inf")


def put(c, side, r, j, x, column=slice(None)):
    """x into key or value j of request r, in one column of all heads or in all of them."""
    c[side][c["table"][r, j // c["page"]].long(), j % c["page"], :, column] = x


def check_tokens(gdn, c, window=0, step=1):
    """Every step-th token against a request of that token alone, by the definition: NaN where that is NaN, infinite
    where that is, and inside the tolerance elsewhere."""
    o, st = pu.run_attention(gdn, c, window)
    assert st == 0
    t = 0
    for r, (kv, m) in enumerate(c["lens"]):
        for u in range(0, m, step):
            one = dict(c, q=c["q"][t + u:t + u + 1], table=c["table"][r:r + 1], lens=[(kv - m + u + 1, 1)])
            ref, tol = (x[0] for x in pu.reference(one, window))
            got, what = o[t + u].double(), f"request {r} token {u}"
            assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
            inf = torch.isinf(ref)
            assert torch.equal(got[inf], ref[inf]), what
            ok = torch.isfinite(ref)
            pu.assert_close(got[ok], ref[ok], tol[ok], what)
        t += m
    return o


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("h_q,h_kv,d,dtype", HEADS)
def test_a_token_of_nan(gdn, h_q, h_kv, d, dtype, window):
    # q, k and v of one token, not the first of its row tile: the ones before it are whole, it and those that see it NaN
    lens = [(200, 40), (129, 129), (1500, 12), (700, 1)]
    c = pu.make_case(lens, h_q, h_kv, d, dtype, page=16, seed=51)
    q = c["q"].clone()
    t = 0
    for r, (kv, m) in enumerate(lens):
        if m > 1:
            u = m // 2 + 1
            q[t + u] = NAN
            put(c, "k", r, kv - m + u, NAN)
            put(c, "v", r, kv - m + u, NAN)
        t += m
    o = check_tokens(gdn, dict(c, q=q), window, step=1 if window else 3)
    assert torch.isnan(o[21]).all() and torch.isfinite(o[20]).all()


@pytest.mark.parametrize("h_q,h_kv,d,dtype", HEADS)
def test_a_score_of_nan_at_a_windows_first_key(gdn, h_q, h_kv, d, dtype):
    # request 0: the first keys that some tokens see; request 1: at a tile's first and last key
    c = pu.make_case([(300, 100), (400, 250)], h_q, h_kv, d, dtype, page=48, seed=52)
    for r, j in ((0, 230), (0, 255), (1, 128), (1, 255)):
        put(c, "k", r, j, NAN, 5)
    put(c, "v", 0, 280, NAN, 3)
    put(c, "v", 1, 390, INF, 4)
    check_tokens(gdn, c, window=60, step=2)


@pytest.mark.parametrize("window", [1, 2])
@pytest.mark.parametrize("h_q,h_kv,d,dtype", HEADS)
def test_scores_of_nan_in_one_of_two_tiles(gdn, h_q, h_kv, d, dtype, window):
    # a row tile whose tokens see one key tile or the other, and all that some of them see is NaN
    lens = [(130, 4), (258, 5), (385, 3)]
    c = pu.make_case(lens, h_q, h_kv, d, dtype, page=16, seed=53)
    for r, j in ((0, 128), (1, 255), (1, 256), (2, 383), (2, 384)):
        put(c, "k", r, j, NAN, 7)
    check_tokens(gdn, c, window)


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("h_q,h_kv,d,dtype", HEADS)
def test_infinite_values(gdn, h_q, h_kv, d, dtype, window):
    lens = [(500, 60), (256, 256), (900, 7)]
    c = pu.make_case(lens, h_q, h_kv, d, dtype, page=32, seed=54, q_gain=0.5)
    for r, (kv, m) in enumerate(lens):
        put(c, "v", r, kv - m + 1, INF, 0)
        put(c, "v", r, kv - m + 3, INF, d - 1)
        put(c, "v", r, kv - m + 4, -INF, d - 1)   # both signs: NaN from here on
        put(c, "v", r, kv - 2, -INF, 33)
    for r, j in ((0, 380), (1, 100)):             # in earlier tokens: all see it, or with a window the first ones do
        put(c, "v", r, j, -INF, 1)
    put(c, "k", 1, 200, -INF, 2)                  # scores of either infinity beside an infinite value
    put(c, "v", 1, 200, INF, 2)
    check_tokens(gdn, c, window, step=3)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("h_q,h_kv,d,dtype", HEADS)
def test_what_is_not_seen_changes_no_bit(gdn, h_q, h_kv, d, dtype, window):
    lens = [(500, 60), (256, 256), (2000, 7), (900, 300)]
    c = pu.make_case(lens, h_q, h_kv, d, dtype, page=32, seed=55)
    want, _ = pu.run_attention(gdn, c, window)
    where = [(0, 450), (0, 499), (1, 127), (1, 128), (2, 1995), (3, 610), (3, 896)]
    for i, (r, j) in enumerate(where):
        put(c, "v", r, j, (NAN, INF, -INF)[i % 3], 3)
        put(c, "k", r, j, (INF, NAN)[i % 2])
    got, st = pu.run_attention(gdn, c, window)
    assert st == 0
    t = 0
    for r, (kv, m) in enumerate(lens):
        pos = kv - m + torch.arange(m, device="cuda")
        sees = torch.zeros(m, dtype=torch.bool, device="cuda")
        for _, j in (x for x in where if x[0] == r):
            sees |= (pos >= j) & ((pos - window < j) if window else True)
        assert sees.any() and not sees.all()
        assert torch.equal(got[t:t + m][~sees], want[t:t + m][~sees])
        assert not torch.isfinite(got[t:t + m][sees]).all(-1).any()
        t += m


@pytest.mark.parametrize("h_q,h_kv,d", [(16, 2, 256), (32, 8, 128), (16, 16, 64)])
def test_long_contexts_behind_values_that_are_not_finite(gdn, h_q, h_kv, d):
    # What it costs goes by the chunk, not by the context: no wait may run out.  (Not split: 80 row items and more.)
    c = pu.make_case([(100000, 1400), (300, 2)], h_q, h_kv, d, page=64, seed=56)
    want, st = pu.run_attention(gdn, c)
    assert st == 0
    put(c, "v", 0, 99000, NAN, 3)
    put(c, "v", 0, 99990, INF, 5)
    got, st = pu.run_attention(gdn, c)
    assert st == 0
    same = torch.ones_like(got, dtype=torch.bool)
    same[400:1400, :, 3] = False
    same[1390:1400, :, 5] = False
    assert torch.equal(got[same], want[same])
    assert torch.isnan(got[400:1400, :, 3]).all() and bool((got[1390:1400, :, 5] == INF).all())
    # all of the chunk after its first token, as a model that has diverged leaves it
    j = torch.arange(98601, 100000, device="cuda")
    for side in "kv":
        c[side][c["table"][0, j // 64].long(), j % 64] = NAN
    got, st = pu.run_attention(gdn, c)
    assert st == 0
    assert torch.equal(got[:1], want[:1]) and torch.equal(got[1400:], want[1400:]) and torch.isnan(got[1:1400]).all()
