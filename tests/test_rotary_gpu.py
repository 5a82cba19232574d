"""gdn_rotary against the rotation by its definition in 64 bits."""
import math

import pytest
import torch

from tests.paged_util import DTYPES, assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def angles(positions, frequencies):
    """In 64 bits: the fraction of a turn is exact in integers."""
    turns = [[(p * (f % (1 << 64))) % (1 << 64) / 2.0 ** 64 for f in frequencies.tolist()] for p in positions.tolist()]
    return torch.tensor(turns, dtype=torch.float64, device="cuda").reshape(len(positions), -1) * (2 * math.pi)


def reference(x, positions, frequencies, interleaved, magnitude):
    """(out, tol): half a step of the type; sine and cosine off by 2^-21 (the fraction of a turn rounded to 24 bits, two
    units of sincospi, the magnitude's product), fp32 sums of two products."""
    rot = 2 * frequencies.numel()
    out, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    angle = angles(positions, frequencies)[:, None]
    cos, sin = angle.cos() * magnitude, angle.sin() * magnitude
    a, b = x[..., at[0]].double(), x[..., at[1]].double()
    out[..., at[0]], out[..., at[1]] = a * cos - b * sin, b * cos + a * sin
    eps = torch.finfo(x.dtype).eps / 2
    small = 2.0 ** -25 if x.dtype == torch.float16 else 0.0  # half of its smallest step
    for s in at:
        tol[..., s] = eps * 1.01 * out[..., s].abs() + (a.abs() + b.abs()) * abs(magnitude) * 2.0 ** -21 + small
    return out, tol


def tensors(T, h_q, h_kv, d, dtype, seed=0):
    """q and k as slices of one projection's output."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((T, h_q + 2 * h_kv, d), generator=gen, device="cuda").to(DTYPES[dtype])
    return qkv[:, :h_q], qkv[:, h_q:h_q + h_kv]


def check(gdn, q, k, positions, freq, interleaved=False, magnitude=1.0, in_place=False):
    wants = [None if x is None else reference(x, positions, freq, interleaved, magnitude) for x in (q, k)]
    if in_place:
        outs = (q, k)
        gdn.gdn_rotary(q, k, positions, freq, interleaved=interleaved, magnitude=magnitude)
    else:
        outs = tuple(None if x is None else torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda") for x in (q, k))
        gdn.gdn_rotary(q, k, positions, freq, *outs, interleaved=interleaved, magnitude=magnitude)
    torch.cuda.synchronize()
    for name, out, want in zip("qk", outs, wants):
        if out is not None:
            assert_close(out, *want, name)
    return outs


SIZES = [(1, 16, 2, 256, 64), (7, 16, 2, 256, 256), (33, 32, 8, 128, 128), (5, 3, 1, 64, 32), (300, 4, 4, 64, 64),
         (9, 5, 1, 80, 20), (6, 2, 2, 80, 48), (4, 1, 1, 2, 2), (11, 2, 1, 100, 16), (3, 7, 7, 1024, 1024), (2000, 12, 4, 128, 96)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,h_q,h_kv,d,rot", SIZES)
def test_rotation(gdn, T, h_q, h_kv, d, rot, interleaved, dtype):
    q, k = tensors(T, h_q, h_kv, d, dtype)
    positions = torch.randint(0, 200000, (T,), device="cuda", dtype=torch.int32)
    freq = gdn.gdn_rotary_frequencies(rot, 10000.0, "linear", 4.0).cuda()
    check(gdn, q, k, positions, freq, interleaved)
    check(gdn, q.clone(), k.clone(), positions, freq, interleaved, magnitude=1.37, in_place=True)
    qkv = torch.cat([q, k], 1)  # slices of one tensor, in place: what lies beside them stays
    keep = qkv.clone()
    check(gdn, qkv[:, :1], None, positions, freq, interleaved, in_place=True)
    assert torch.equal(qkv[:, 1:], keep[:, 1:]) and torch.equal(qkv[..., rot:], keep[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(gdn, interleaved):
    edge = [0, 1, -1, 2 ** 24 + 1, 10 ** 6, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31, -12345]
    positions = torch.tensor(edge, dtype=torch.int32, device="cuda")
    q, k = tensors(len(edge), 4, 2, 128, "fp16", seed=1)
    for scaling, factor in (("none", 1.0), ("ntk", 8.0), ("yarn", 32.0)):
        freq = gdn.gdn_rotary_frequencies(128, 10000.0, scaling, factor, original_length=4096).cuda()
        check(gdn, q, k, positions, freq, interleaved)
    # a turn backwards undoes one forwards, up to the roundings on the way
    there, _ = check(gdn, q, None, positions[1:2].expand(len(edge)).contiguous(), freq)
    back, _ = check(gdn, there, None, positions[2:3].expand(len(edge)).contiguous(), freq)
    assert (back.double() - q.double()).abs().max() <= 4 * 2.0 ** -11 * q.abs().max()


@pytest.mark.parametrize("interleaved", [False, True])
def test_any_alignment_gives_the_same_bits(gdn, interleaved):
    # 16-byte pieces, and pairs where addresses or strides do not allow them
    q, k = tensors(37, 6, 2, 64, "bf16", seed=2)
    positions = torch.arange(37, device="cuda", dtype=torch.int32) * 1001
    freq = gdn.gdn_rotary_frequencies(32).cuda()
    want_q, want_k = check(gdn, q, k, positions, freq, interleaved)
    for pad, start in ((8, 0), (3, 0), (8, 1), (5, 2)):
        wide = torch.zeros((37, 8, 64 + pad + start), dtype=torch.bfloat16, device="cuda")
        view = wide[..., start:start + 64]
        view.copy_(torch.cat([q, k], 1))
        got = check(gdn, view[:, :6], view[:, 6:], positions, freq, interleaved)
        assert torch.equal(got[0], want_q) and torch.equal(got[1], want_k)
        check(gdn, view[:, :6], view[:, 6:], positions, freq, interleaved, in_place=True)
        assert torch.equal(view[:, :6], want_q) and torch.equal(view[:, 6:], want_k)
        assert not wide[..., :start].any() and not wide[..., start + 64:].any()


def test_inputs_shared_by_heads(gdn):
    x = torch.randn(20, 1, 128, device="cuda").bfloat16()
    positions = torch.arange(20, device="cuda", dtype=torch.int32)
    freq = gdn.gdn_rotary_frequencies(128).cuda()
    q, _ = check(gdn, x.expand(20, 5, 128), None, positions, freq)
    assert torch.equal(q[:, 0], q[:, 4])


def test_a_token_does_not_depend_on_the_others(gdn):
    q, k = tensors(3000, 8, 2, 128, "bf16", seed=3)
    positions = torch.randint(0, 100000, (3000,), device="cuda", dtype=torch.int32)
    freq = gdn.gdn_rotary_frequencies(128).cuda()
    all_q, all_k = (torch.empty_like(x) for x in (q, k))
    gdn.gdn_rotary(q, k, positions, freq, all_q, all_k)
    for t in (0, 1, 1499, 2999):
        one = [torch.empty_like(x[t:t + 1]) for x in (q, k)]
        gdn.gdn_rotary(q[t:t + 1], k[t:t + 1], positions[t:t + 1], freq, *one)
        assert torch.equal(one[0][0], all_q[t]) and torch.equal(one[1][0], all_k[t])


def test_values_that_are_not_finite_stay_in_their_pair(gdn):
    q, _ = tensors(4, 2, 1, 64, "bf16", seed=4)
    q = q.clone()
    positions = torch.arange(4, device="cuda", dtype=torch.int32) + 5
    freq = gdn.gdn_rotary_frequencies(32).cuda()
    want = torch.empty_like(q)
    gdn.gdn_rotary(q, None, positions, freq, want)
    q[1, 0, 3], q[2, 1, 40] = float("nan"), float("inf")
    got = torch.empty_like(q)
    gdn.gdn_rotary(q, None, positions, freq, got)
    assert torch.isnan(got[1, 0, 3]) and torch.isnan(got[1, 0, 19]) and got[2, 1, 40] == float("inf")
    for t, h, i in ((1, 0, 3), (1, 0, 19), (2, 1, 40)):
        got[t, h, i] = want[t, h, i]
    assert torch.equal(got, want)


def test_capture_on_another_stream(gdn):
    q, k = tensors(50, 4, 1, 128, "bf16", seed=5)
    positions = torch.arange(50, device="cuda", dtype=torch.int32)
    freq = gdn.gdn_rotary_frequencies(64).cuda()
    out = [torch.empty_like(x) for x in (q, k)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_rotary(q, k, positions, freq, *out)
    positions += 1000
    g.replay()
    want = [torch.empty_like(x) for x in (q, k)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gdn.gdn_rotary(q, k, positions, freq, *want, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    gdn.gdn_rotary(q[:0], k[:0], positions[:0], freq)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pad,start", [(4, 4), (2, 2), (6, 0), (4, 0), (1, 0)])
def test_pieces_of_any_width_give_the_same_bits(gdn, pad, start, interleaved):
    q, k = tensors(41, 5, 2, 96, "fp16", seed=6)
    positions = torch.arange(41, device="cuda", dtype=torch.int32) * 777
    freq = gdn.gdn_rotary_frequencies(64).cuda()
    want_q, want_k = check(gdn, q, k, positions, freq, interleaved)
    wide = torch.zeros((41, 7, 96 + pad + start), dtype=torch.float16, device="cuda")
    view = wide[..., start:start + 96]
    view.copy_(torch.cat([q, k], 1))
    got = check(gdn, view[:, :5], view[:, 5:], positions, freq, interleaved)  # from there, into 16-byte rows
    assert torch.equal(got[0], want_q) and torch.equal(got[1], want_k)
    check(gdn, view[:, :5], view[:, 5:], positions, freq, interleaved, in_place=True)
    assert torch.equal(view[:, :5], want_q) and torch.equal(view[:, 5:], want_k)
    assert not wide[..., :start].any() and not wide[..., start + 96:].any()


@pytest.mark.parametrize("d,rot", [(80, 20), (100, 16), (128, 128), (96, 32), (70, 68)])
def test_many_tokens(gdn, d, rot):
    T = 40000
    q, k = tensors(T, 3, 1, d, "bf16", seed=7)
    positions = torch.randint(0, 1 << 20, (T,), device="cuda", dtype=torch.int32)
    freq = gdn.gdn_rotary_frequencies(rot).cuda()
    outs = [torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda") for x in (q, k)]
    gdn.gdn_rotary(q, k, positions, freq, *outs)
    at = torch.cat([torch.arange(200), torch.randint(0, T, (200,)), torch.arange(T - 200, T)]).cuda()
    for x, out in zip((q, k), outs):
        assert torch.isfinite(out).all()
        assert_close(out[at], *reference(x[at], positions[at], freq, False, 1.0))
        assert torch.equal(out[..., rot:], x[..., rot:])
