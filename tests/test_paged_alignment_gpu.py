"""The paged calls on buffers that start at a multiple of 16 bytes but not of 32: what the contract asks for."""
import pytest
import torch

from tests import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def at_16(t):
    """The same values in a dense tensor 8 elements into its buffer."""
    buf = torch.full((t.numel() + 16,), float("nan"), dtype=t.dtype, device=t.device)
    out = buf[8:8 + t.numel()].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 32 == 16
    return out, buf


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("h_q,h_kv,d", [(16, 2, 256), (8, 2, 128), (5, 1, 128), (6, 2, 64), (3, 3, 64)])
def test_output_and_inputs_at_16_bytes(gdn, h_q, h_kv, d, dtype):
    # whole and split requests, one and two row tiles, tokens that see nothing, padding
    lens = [(300, 300), (3000, 1), (1153, 200), (5, 9), (64, 3), (0, 2)]
    c = pu.make_case(lens, h_q, h_kv, d, dtype, page=32, seed=41, pad=3)
    want, st = pu.run_attention(gdn, c)
    assert st == 0
    q, k, v = (at_16(c[x].contiguous())[0] for x in "qkv")
    o, buf = at_16(torch.full_like(want, float("nan")))
    n = gdn.gdn_paged_attention_workspace_bytes(h_q, h_kv, d, len(lens), q.shape[0], c["table"].shape[1] * 32)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_paged_attention(q, k, v, c["table"], c["cu"], c["kv"], o, workspace=ws, dev_status=word)
    assert word.item() == 0 and torch.equal(o, want)
    assert torch.isnan(buf[:8]).all() and torch.isnan(buf[8 + o.numel():]).all()


def test_write_at_16_bytes(gdn):
    gen = torch.Generator(device="cuda").manual_seed(42)
    k, v = (at_16(torch.randn((37, 2, 64), generator=gen, device="cuda").bfloat16())[0] for _ in range(2))
    kc, vc = (at_16(torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda"))[0] for _ in range(2))
    slots = torch.randperm(64, generator=gen, device="cuda")[:37].to(torch.int32)
    gdn.gdn_paged_kv_write(k, v, kc, vc, slots)
    for got, new in ((kc, k), (vc, v)):
        want = torch.zeros_like(got)
        want[slots.long() // 16, slots.long() % 16] = new
        assert torch.equal(got, want)
