"""Small fp16 weights of a long context: a tail that holds a part of the sum of weights holds it in the result too."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


@pytest.mark.parametrize("h_q,h_kv,d,m", [(80, 80, 64, 256), (80, 80, 128, 256), (80, 80, 256, 128), (80, 10, 64, 320)])
def test_a_tail_of_small_weights(gdn, h_q, h_kv, d, m):
    # Key 0 has all but a sliver of the weight and a value of zero; each of the n others has 2^-25.5 of its weight and a
    # value of v: the output is n w v / (1 + n w).  (80 row items and more: no split, whose parts have maxima of their own.)
    n, page = 20000, 1088
    pages = -(-(n + m) // page)
    k, v = (torch.zeros((pages, page, h_kv, d), dtype=torch.float16, device="cuda") for _ in range(2))
    v[..., :] = torch.linspace(1, 2, d, device="cuda").half()
    k[0, 0, :, 0] = 8.0
    v[0, 0] = 0.0
    q = torch.zeros((m, h_q, d), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    scale = 25.5 * math.log(2) / 8
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    kv = torch.tensor([n + m], dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    ws = torch.empty(gdn.gdn_paged_attention_workspace_bytes(h_q, h_kv, d, 1, m, n + m), dtype=torch.uint8, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_paged_attention(q, k, v, table, cu, kv, o, scale=scale, max_kv_len=n + m, workspace=ws, dev_status=word)
    assert word.item() == 0
    tail = (n + torch.arange(m, device="cuda", dtype=torch.float64)) * 2.0 ** -25.5
    values = v[1, 1, 0].double()
    want = (tail / (1 + tail))[:, None, None] * values
    # Half a step of the output and of each weight.  Weights are held as 2^7 of the formula's: under fp16's smallest
    # normal, half of its smallest step is 2^-25 / 2^7 of the largest weight each.  2^-12: the scores' and the sums' 32 bits
    # (25.5 x 2^-24 in the exponent; 1400 partial sums of the product, each off by 2^-23 at most).
    n_seen = (n + torch.arange(m, device="cuda", dtype=torch.float64))[:, None, None]
    tol = want * (2 * 2.0 ** -11 + 2.0 ** -12) + n_seen * 2.0 ** -32 * values
    err = (o.double() - want).abs()
    assert bool((err <= tol).all()), (err / want).max().item()
