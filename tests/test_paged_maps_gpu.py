"""The step's maps and the K/V write over the paged cache, and the three paged calls together."""
import random

import pytest
import torch

from tests import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_serving_gdn_gb300 as g
    g.load_library()
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_maps(gdn, ctx, new, table, page, num_pages, capacity, free=None, head=0, in_place=False):
    n = len(ctx)
    dev_table = i32(table).reshape(n, -1)
    cu, kv = torch.full((n + 1,), 77, dtype=torch.int32, device="cuda"), torch.full((n,), 77, dtype=torch.int32, device="cuda")
    slots, pos = (torch.full((capacity,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    st, h0 = i32([0]), i32([head])
    h1 = h0 if in_place else i32([-5])
    kw = {} if free is None else dict(free_pages=i32(free), free_head=h0, free_head_out=h1)
    gdn.gdn_paged_maps(i32(ctx), i32(new), dev_table, page, num_pages, cu, kv, slots, pos, dev_status=st, **kw)
    want = [list(r) for r in table]
    w_cu, w_kv, w_slots, w_pos, w_head, w_st = pu.maps_reference(ctx, new, want, page, num_pages, capacity, free, head)
    assert cu.tolist() == w_cu and kv.tolist() == w_kv
    assert slots.tolist() == w_slots and pos.tolist() == w_pos
    assert dev_table.tolist() == want
    if free is not None:
        assert h1.item() == w_head
        assert in_place or h0.item() == head
    assert st.item() == w_st


def random_step(rng, n, page, max_new, max_ctx, spare=0, pad=0, decodes=0):
    ctx = [rng.choice([0, page, rng.randint(0, max_ctx)]) for _ in range(n)]
    new = [1 if i < decodes else rng.choice([0, 1, rng.randint(0, max_new)]) for i in range(n)]
    width = max(pu.ceil(c + m, page) for c, m in zip(ctx, new)) + 1
    total = sum(pu.ceil(c + m, page) for c, m in zip(ctx, new))
    ids = list(range(total + 20))
    rng.shuffle(ids)
    table = []
    for c in ctx:
        have = pu.ceil(c, page)
        table.append([ids.pop() for _ in range(have)] + [-1] * (width - have))
    head = rng.randint(0, 5)
    need = sum(pu.ceil(c + m, page) - pu.ceil(c, page) for c, m in zip(ctx, new))
    free = ids[:max(0, head + need + spare)]
    return ctx, new, table, page, total + 20, sum(new) + pad, free, head


@pytest.mark.parametrize("n,page,max_new,max_ctx", [(1, 16, 1, 50), (1, 1, 9, 9), (7, 16, 40, 100), (33, 48, 300, 2000),
                                                    (1023, 16, 3, 70), (1024, 1088, 2, 5000), (1025, 64, 5, 300),
                                                    (3000, 16, 20, 64), (5, 1088, 9000, 5000)])
def test_maps(gdn, n, page, max_new, max_ctx):
    rng = random.Random(n * page)
    check_maps(gdn, *random_step(rng, n, page, max_new, max_ctx, pad=rng.randint(0, 40)))
    check_maps(gdn, *random_step(rng, n, page, max_new, max_ctx, spare=3, decodes=n // 2), in_place=True)


def test_maps_long_prompt_among_decodes(gdn):
    rng = random.Random(5)
    ctx = [rng.randint(0, 300) for _ in range(40)] + [17]
    new = [1] * 40 + [70000]
    page = 16
    width = pu.ceil(70017, page)
    table = [[1000 * i + j for j in range(pu.ceil(c, page))] + [-1] * (width - pu.ceil(c, page)) for i, c in enumerate(ctx)]
    free = list(range(50000, 50000 + 4500))
    check_maps(gdn, ctx, new, table, page, 60000, sum(new) + 5, free, 3)


def test_maps_without_a_free_list(gdn):
    check_maps(gdn, [5, 0, 31], [3, 16, 1], [[4, -1], [2, 9], [1, 0]], 16, 10, 25)


def test_maps_when_pages_run_out(gdn):
    # the first two are served, the third and every later one that needs a page are not; the fourth needs none
    ctx, new = [0, 16, 30, 3, 0, 16], [20, 1, 40, 2, 1, 1]
    table = [[-1] * 6, [7] + [-1] * 5, [8, 9] + [-1] * 4, [10] + [-1] * 5, [-1] * 6, [11] + [-1] * 5]
    check_maps(gdn, ctx, new, table, 16, 100, sum(new) + 2, [20, 21, 22, 23], 1, in_place=True)
    check_maps(gdn, ctx, new, table, 16, 100, sum(new), [], 0)


def test_maps_refusals(gdn):
    table = [[3, -1, -1]] * 6
    big = 2 ** 31 - 1
    check_maps(gdn, [5, -1, 5, big, 40, 0], [2, 3, -4, 5, 20, 1], table, 16, 50, 40, list(range(10, 20)), 0)
    check_maps(gdn, [0, 0, 0], [10, 10, 10], table[:3], 16, 50, 25, list(range(10, 20)), 0)  # tokens past the capacity
    check_maps(gdn, [0, 0], [10, 0], table[:2], 16, 50, 12, list(range(10, 20)), -3)          # a head before the list
    check_maps(gdn, [5, 0], [2, 3], [[-1, -1], [3, 1]], 16, 50, 5, [60, 61], 0)               # page ids out of range


def test_maps_of_no_request(gdn):
    cu, slots, pos = i32([9]), i32([9, 9]), i32([9, 9])
    gdn.gdn_paged_maps(i32([]), i32([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 16, 4, cu, i32([]), slots, pos)
    assert cu.tolist() == [0] and slots.tolist() == [-1, -1] and pos.tolist() == [0, 0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
@pytest.mark.parametrize("tokens,h,d,page", [(1, 2, 256, 1088), (257, 3, 64, 48), (4000, 8, 128, 16), (50, 1, 128, 32)])
def test_write(gdn, tokens, h, d, page, layout, dtype):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    dt = pu.DTYPES[dtype]
    pages = pu.ceil(tokens, page) + 2
    k, v = pu.make_cache(gen, pages, page, h, d, dt, layout)
    qkv = torch.randn((tokens, 4 * h, d), generator=gen, device="cuda").to(dt)
    src_k, src_v = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:tokens].to(torch.int32)
    slots[::7] = -1
    bad = 0
    if tokens > 10:
        slots[3] = pages * page
        bad = gdn.GDN_DEV_BAD_SLOT
    want_k, want_v = k.clone(), v.clone()
    live = (slots >= 0) & (slots < pages * page)
    at = slots[live].long()
    want_k[at // page, at % page], want_v[at // page, at % page] = src_k[live], src_v[live]
    st = i32([0])
    gdn.gdn_paged_kv_write(src_k, src_v, k, v, slots, dev_status=st)
    assert st.item() == bad
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def test_write_past_32_bits(gdn):
    d, h, page = 128, 8, 1088
    pages = (1 << 31) // (page * h * d) + 3
    k = torch.empty((pages, page, h, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    new = torch.randn((2, 4, h, d), device="cuda").bfloat16()
    slots = i32([pages * page - 1, 0, (pages - 1) * page, -1])
    gdn.gdn_paged_kv_write(new[0], new[1], k, v, slots)
    assert torch.equal(k[-1, -1], new[0, 0]) and torch.equal(v[-1, 0], new[1, 2]) and torch.equal(k[0, 0], new[0, 1])


def test_steps_of_a_served_batch(gdn):
    """Prompts in chunks, then decodes, each step from its lengths alone: every token's output is that of one
    attention over the tokens so far, whatever pages the steps took."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    h_q, h_kv, d, page, n = 8, 2, 128, 16, 3
    steps = [[40, 0, 1], [70, 33, 0], [1, 100, 1], [1, 1, 5], [1, 1, 1]]
    total = [sum(s[i] for s in steps) for i in range(n)]
    data = [torch.randn((t, h_q + 2 * h_kv, d), generator=gen, device="cuda").bfloat16() for t in total]
    pages = sum(pu.ceil(t, page) for t in total) + 4
    k, v = pu.make_cache(gen, pages, page, h_kv, d, torch.bfloat16, "hnd")
    k.fill_(float("nan")), v.fill_(float("nan"))
    table = torch.full((n, 16), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    head, st = i32([0]), i32([0])
    ctx, outs = [0] * n, [[] for _ in range(n)]
    for new in steps:
        T = sum(new) + 2
        cu, kv, slots, pos = i32([0] * (n + 1)), i32([0] * n), i32([0] * T), i32([0] * T)
        gdn.gdn_paged_maps(i32(ctx), i32(new), table, page, pages, cu, kv, slots, pos, free_pages=free,
                           free_head=head, dev_status=st)
        rows = torch.cat([data[i][ctx[i]:ctx[i] + new[i]] for i in range(n)] + [torch.full_like(data[0][:2], float("nan"))])
        gdn.gdn_paged_kv_write(rows[:, h_q:h_q + h_kv], rows[:, h_q + h_kv:], k, v, slots, dev_status=st)
        o = torch.empty((T, h_q, d), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(gdn.gdn_paged_attention_workspace_bytes(h_q, h_kv, d, n, T, 256), dtype=torch.uint8, device="cuda")
        gdn.gdn_paged_attention(rows[:, :h_q], k, v, table, cu, kv, o, workspace=ws, dev_status=st)
        at = 0
        for i in range(n):
            outs[i].append(o[at:at + new[i]])
            at += new[i]
            ctx[i] += new[i]
    assert st.item() == 0 and head.item() == sum(pu.ceil(t, page) for t in total)
    whole = {"q": torch.cat([x[:, :h_q] for x in data]), "k": k, "v": v, "table": table, "page": page,
             "lens": [(t, t) for t in total]}
    ref, tol = pu.reference(whole)
    pu.assert_close(torch.cat([torch.cat(x) for x in outs]), ref, tol)


def test_a_captured_step_replays_for_other_lengths(gdn):
    gen = torch.Generator(device="cuda").manual_seed(4)
    h_q, h_kv, d, page, n, T, width = 8, 2, 64, 16, 6, 40, 20
    pages = 80
    k, v = pu.make_cache(gen, pages, page, h_kv, d, torch.bfloat16, "nhd")
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    start_table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    for i in range(n):
        start_table[i, :8] = perm[8 * i:8 * i + 8]
    free = perm[8 * n:].contiguous()
    table, head, st = start_table.clone(), i32([0]), i32([0])
    ctx, new = i32([0] * n), i32([0] * n)
    cu, kv, slots, pos = i32([0] * (n + 1)), i32([0] * n), i32([0] * T), i32([0] * T)
    rows = torch.randn((T, h_q + 2 * h_kv, d), generator=gen, device="cuda").bfloat16()
    o = torch.empty((T, h_q, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gdn.gdn_paged_attention_workspace_bytes(h_q, h_kv, d, n, T, width * page), dtype=torch.uint8, device="cuda")

    def step(stream):
        gdn.gdn_paged_maps(ctx, new, table, page, pages, cu, kv, slots, pos, free_pages=free, free_head=head,
                           dev_status=st, stream=stream)
        gdn.gdn_paged_kv_write(rows[:, h_q:h_q + h_kv], rows[:, h_q + h_kv:], k, v, slots, dev_status=st, stream=stream)
        gdn.gdn_paged_attention(rows[:, :h_q], k, v, table, cu, kv, o, workspace=ws, dev_status=st, stream=stream)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for c, m in [([3, 100, 128, 0, 7, 64], [1, 1, 1, 1, 1, 1]), ([128, 0, 60, 5, 0, 100], [9, 0, 20, 1, 4, 3]),
                 ([128] * 6, [1, 0, 0, 0, 0, 17])]:
        table.copy_(start_table), head.zero_(), ctx.copy_(i32(c)), new.copy_(i32(m))
        graph.replay()
        torch.cuda.synchronize()
        assert st.item() == 0
        got = o.clone()
        want = {"q": rows[:, :h_q], "k": k, "v": v, "table": table, "page": page, "lens": [(a + b, b) for a, b in zip(c, m)]}
        ref, tol = pu.reference(want)
        pu.assert_close(got, ref, tol)
        table.copy_(start_table), head.zero_()
        step(None)
        torch.cuda.synchronize()
        assert torch.equal(o, got)
