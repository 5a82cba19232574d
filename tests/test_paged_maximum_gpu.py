"""The running maximum of the paged attention: scores that make it move late, often, and in some rows of a warp only."""
import pytest
import torch

from tests import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def rising(lens, h_q, h_kv, d, dtype, gains, seed):
    """Keys whose first element grows (request 0) or falls (request 1) along the context, all else small; query row
    (token t, head h) takes it with gains[(t + h) % len(gains)]."""
    c = pu.make_case(lens, h_q, h_kv, d, dtype, page=32, seed=seed, q_gain=0.05)
    for r, (kv, _) in enumerate(lens):
        j = torch.arange(kv, device="cuda")
        page, row = c["table"][r, j // 32].long(), j % 32
        c["k"][page, row] *= 0.02
        x = (j if r % 2 == 0 else kv - j) / 10.0
        c["k"][page, row, :, 0] = x[:, None].to(c["k"].dtype)
    T = c["q"].shape[0]
    which = torch.arange(T, device="cuda")[:, None] + torch.arange(h_q, device="cuda")
    c["q"][..., 0] = torch.tensor(gains, device="cuda", dtype=c["q"].dtype)[which % len(gains)]
    return c


# gains: all rows move in every tile; every third row does; one in seven, the others down or not at all
@pytest.mark.parametrize("gains", [(4.0,), (4.0, 0.0, 0.0), (6.0, 0.0, -4.0, 0.1, 0.0, -0.1, 0.0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("h_q,h_kv,d", [(4, 2, 64), (8, 2, 128), (5, 1, 128), (2, 2, 128), (4, 2, 256)])
def test_rising_scores(gdn, h_q, h_kv, d, dtype, gains):
    c = rising([(900, 130), (900, 1), (1000, 300), (700, 5), (1300, 1)], h_q, h_kv, d, dtype, gains, seed=61)
    o, st = pu.run_attention(gdn, c)
    assert st == 0
    ref, tol = pu.reference(c)
    pu.assert_close(o, ref, tol)


@pytest.mark.parametrize("h_q,h_kv,d", [(32, 16, 64), (32, 8, 128), (16, 8, 256)])
def test_rising_scores_of_whole_requests_with_a_window(gdn, h_q, h_kv, d):
    # (80 row items and more: not split)
    c = rising([(700, 700), (650, 640)], h_q, h_kv, d, "bf16", (4.0, 0.0, -3.0), seed=62)
    o, st = pu.run_attention(gdn, c, window=400)
    assert st == 0
    ref, tol = pu.reference(c, 400)
    pu.assert_close(o, ref, tol)


@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (2, 2, 128)])
def test_a_row_does_not_depend_on_how_its_neighbours_maxima_move(gdn, h_q, h_kv, d):
    lens = [(900, 130), (900, 1), (1000, 300)]
    a = rising(lens, h_q, h_kv, d, "bf16", (4.0, 0.0, 0.0, 0.5), seed=63)
    b = rising(lens, h_q, h_kv, d, "bf16", (4.0, 3.0, -2.0, 0.5), seed=63)
    (x, _), (y, _) = pu.run_attention(gdn, a), pu.run_attention(gdn, b)
    which = (torch.arange(x.shape[0], device="cuda")[:, None] + torch.arange(h_q, device="cuda")) % 4
    same = (which == 0) | (which == 3)
    assert torch.equal(x[same], y[same])
