"""gdn_rotary of q or k alone."""
import pytest
import torch

from tests.test_rotary_gpu import gdn, reference, tensors  # noqa: F401
from tests.paged_util import assert_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,d,rot", [(1, 128, 64), (700, 64, 64), (9, 80, 20)])
def test_one_side_gives_the_bits_of_both(gdn, T, d, rot, in_place):  # noqa: F811
    q, k = tensors(T, 4, 2, d, "bf16", seed=8)
    positions = torch.randint(0, 100000, (T,), device="cuda", dtype=torch.int32)
    freq = gdn.gdn_rotary_frequencies(rot).cuda()
    both = [torch.empty_like(x) for x in (q, k)]
    gdn.gdn_rotary(q, k, positions, freq, *both)
    assert_close(both[1], *reference(k, positions, freq, False, 1.0))
    keep = q.clone()
    if in_place:
        out = k
        gdn.gdn_rotary(None, k, positions, freq)
    else:
        out = torch.empty_like(k)
        gdn.gdn_rotary(None, k, positions, freq, k_out=out)
    assert torch.equal(out, both[1]) and torch.equal(q, keep)
    out = torch.empty_like(q)
    gdn.gdn_rotary(q, None, positions, freq, q_out=out)
    assert torch.equal(out, both[0])
