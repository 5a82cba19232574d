"""Cases of the paged-attention operators: the maps of a step, the K/V write, and attention over the paged cache.

``run`` computes an operator in its plain form (elementary torch operations) or, with ``own`` set, through the
framework's entry points.  A case is a plain dict; ``prepare`` turns it into the tensors a serving program holds
before the step.
"""
from __future__ import annotations

import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# Request lengths are derived from the case's own "lens_seed", so that `work`
# and `prepare` agree on them; the values of the tensors come from the seed
# given to `prepare`.

def _attn(name, n, new_lo, new_hi, ctx_lo, ctx_hi, h_q, h_kv, d, dtype, page, window=0, decodes=0, layout="nhd",
          lens_seed=0):
    """n requests of new_lo..new_hi new tokens on ctx_lo..ctx_hi cached ones, `decodes` of them single tokens."""
    return {"name": name, "op": "attention", "n": n, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "h_q": h_q, "h_kv": h_kv, "d": d, "dtype": dtype, "page": page, "window": window,
            "decodes": decodes, "layout": layout, "lens_seed": lens_seed}


def _maps(name, n, new_lo, new_hi, ctx_lo, ctx_hi, page, decodes=0, pad=0, lens_seed=0):
    return {"name": name, "op": "maps", "n": n, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "page": page, "decodes": decodes, "pad": pad, "lens_seed": lens_seed}


def _write(name, tokens, h_kv, d, dtype, page, layout="nhd", pad=0):
    return {"name": name, "op": "write", "tokens": tokens, "h_kv": h_kv, "d": d, "dtype": dtype, "page": page,
            "layout": layout, "pad": pad}


def listed():
    return [
        # the step metadata of a small decode batch, padded to the captured graph's size
        _maps("maps_decode_8", 8, 1, 1, 100, 4000, 16, pad=8),
        # a large continuous batch: 1000 decode rows and 24 prompt chunks on prefix-cache blocks of 1088 tokens
        _maps("maps_mixed_1024", 1024, 900, 4096, 0, 20000, 1088, decodes=1000),
        # K/V of one decode step, 256 rows
        _write("write_decode_256", 256, 2, 256, "bf16", 1088, pad=3),
        # K/V of a long prompt chunk, head-major pages
        _write("write_chunk_32768", 32768, 8, 128, "fp16", 16, layout="hnd"),
        # one user's next token: nothing but latency
        _attn("attn_one_token", 1, 1, 1, 1058, 1058, 16, 2, 256, "bf16", 64),
        # a decode step of 256 ragged rows on 1088-token blocks
        _attn("attn_decode_256", 256, 1, 1, 31, 4095, 16, 2, 256, "bf16", 1088, lens_seed=1),
        # few very long contexts, small pages
        _attn("attn_decode_long", 8, 1, 1, 100000, 131071, 32, 8, 128, "fp16", 16, lens_seed=2),
        # four drafted tokens to verify per row, one K/V head per query head
        _attn("attn_verify_4", 64, 4, 4, 2000, 8000, 16, 16, 64, "bf16", 32, lens_seed=3),
        # fresh prompts of 100 to 2000 tokens
        _attn("attn_prompts_8", 8, 116, 2000, 0, 0, 16, 2, 256, "bf16", 1088, lens_seed=4),
        # prompt chunks of 2048 tokens late in a 32768-token context
        _attn("attn_chunk_late", 2, 2048, 2048, 32000, 32768, 16, 2, 256, "bf16", 1088, lens_seed=5),
        # one fresh prompt of 8192 tokens
        _attn("attn_prompt_8192", 1, 8192, 8192, 0, 0, 32, 8, 128, "fp16", 16, layout="hnd"),
        # a mixed step with a sliding window: 60 decode rows and 4 chunks, three query heads per K/V head
        _attn("attn_mixed_window", 64, 300, 1500, 0, 6000, 12, 4, 64, "fp16", 48, window=1024, decodes=60, lens_seed=6),
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm of lo..hi, odd values included."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random())) + rng.randint(0, 1)))


def draw(rng: random.Random):
    kind = rng.choice(["maps", "write", "decode", "decode", "verify", "prompt", "chunk", "mixed"])
    seed = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 48, 64, 128, 256, 1088])
    if kind == "maps":
        n = _log_int(rng, 1, 1024)
        chunks = rng.randint(0, min(n, 24))
        return {**_maps("", n, _log_int(rng, 2, 900), 4096, 0, _log_int(rng, 64, 20000), page, decodes=n - chunks,
                        pad=rng.choice([0, 0, rng.randint(1, 64)]), lens_seed=seed)}
    h_kv, group, d = rng.choice([(2, 8, 256), (4, 4, 256), (2, 4, 256), (8, 4, 128), (4, 8, 128), (4, 5, 128),
                                 (16, 1, 128), (16, 1, 64), (4, 3, 64), (1, 16, 64), (8, 2, 64)])
    dtype = rng.choice(["bf16", "fp16"])
    layout = rng.choice(["nhd", "hnd"])
    if kind == "write":
        return _write("", _log_int(rng, 1, 32768 * 1024 // (h_kv * d)), h_kv, d, dtype, page, layout,
                      pad=rng.randint(0, 9))
    window = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
    args = dict(window=window, layout=layout, lens_seed=seed)
    heads = (group * h_kv, h_kv, d, dtype, page)
    if kind == "decode":
        hi = _log_int(rng, 16, 131072)
        # the cache stays within the largest listed one (about 4.3 GB)
        n = _log_int(rng, 1, max(1, min(512, (1 << 30) // (hi * h_kv * d))))
        return _attn("", n, 1, 1, rng.randint(0, hi // 2), hi, *heads, **args)
    if kind == "verify":
        hi = _log_int(rng, 16, 32768)
        n = _log_int(rng, 1, max(1, min(128, (1 << 29) // (hi * h_kv * d))))
        return _attn("", n, 2, rng.randint(2, 9), 0, hi, *heads, **args)
    # products of at most about the largest listed case's: 2 x 2048 tokens x 34000 keys x 16 heads x 256
    budget = 2 * 2048 * 34000 * 16 * 256 // (group * h_kv * d)
    if kind == "prompt":
        new = _log_int(rng, 17, 8192)
        n = _log_int(rng, 1, max(1, min(16, budget // (new * new))))
        return _attn("", n, max(1, new // 8), new, 0, 0, *heads, **args)
    ctx = _log_int(rng, 64, 65536)
    new = _log_int(rng, 17, max(18, min(4096, budget // (ctx + 4096))))
    if kind == "chunk":
        n = _log_int(rng, 1, max(1, min(8, budget // (new * (ctx + new)))))
        return _attn("", n, max(1, new // 2), new, ctx // 2, ctx, *heads, **args)
    ctx = min(ctx, 16384)
    n = rng.randint(3, 64)
    return _attn("", n, max(1, new // 4), min(new, 2048), 0, ctx, *heads, decodes=n - rng.randint(1, 2), **args)


def _lens(case):
    """Host lists (context lengths, new lengths) of the case's requests, decode rows first."""
    rng = random.Random(case["lens_seed"] * 1000003 + case["n"])
    ctx, new = [], []
    for i in range(case["n"]):
        ctx.append(rng.randint(case["ctx_lo"], case["ctx_hi"]))
        new.append(1 if i < case["decodes"] else rng.randint(case["new_lo"], case["new_hi"]))
    return ctx, new


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _cache(gen, pages, page, h, d, dtype, layout):
    """A K or V cache viewed as [pages][page][h][d]; the "hnd" layout holds its pages head by head."""
    shape = (pages, page, h, d) if layout == "nhd" else (pages, h, page, d)
    t = torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[dtype])
    return t if layout == "nhd" else t.permute(0, 2, 1, 3)


def _table(gen, counts, width, pages):
    """Block table [n][width] with counts[i] pages of a random permutation per request, -1 beyond; the pages left."""
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda")
    cnt = torch.tensor(counts, device="cuda")
    first = torch.cumsum(cnt, 0) - cnt
    col = torch.arange(width, device="cuda")
    live = col[None, :] < cnt[:, None]
    table[live] = perm[(first[:, None] + col[None, :])[live]]
    return table, perm[sum(counts):].contiguous()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "maps":
        ctx, new = _lens(case)
        # other seeds are other steps of the same batch: the contexts move on by up to a page
        shift = random.Random(seed).randrange(case["page"])
        ctx = [c + shift for c in ctx]
        P = case["page"]
        have = [_ceil(c, P) for c in ctx]
        total = [_ceil(c + m, P) for c, m in zip(ctx, new)]
        # sizes that hold every shift, so that all seeds' steps have the same shapes
        most = [_ceil(c - shift + P + m, P) for c, m in zip(ctx, new)]
        s["num_pages"] = sum(most) + 17
        s["table"], spare = _table(gen, have, max(most) + 1, s["num_pages"])
        fresh = sum(total) - sum(have)
        # the free list: five pages taken by earlier steps, what this step needs and a few more
        s["free"] = spare[:fresh + 17].clone()
        s["ctx"], s["new"], s["head"] = _i32(ctx), _i32(new), _i32([5])
        T = sum(new) + case["pad"]
        n = case["n"]
        s["cu"], s["kv"], s["head_out"] = _i32([0] * (n + 1)), _i32([0] * n), _i32([0])
        s["slots"], s["pos"] = _i32([0] * T), _i32([0] * T)
        return s
    dtype = DTYPES[case["dtype"]]
    P, h_kv, d = case["page"], case["h_kv"], case["d"]
    if case["op"] == "write":
        T = case["tokens"]
        pages = _ceil(T, P) + 3
        # k and v are slices of one projection's output, as a layer has them
        qkv = torch.randn((T, 4 * h_kv, d), generator=gen, device="cuda", dtype=dtype)
        s["k"], s["v"] = qkv[:, 2 * h_kv:3 * h_kv], qkv[:, 3 * h_kv:]
        s["kc"] = _cache(gen, pages, P, h_kv, d, case["dtype"], case["layout"])
        s["vc"] = _cache(gen, pages, P, h_kv, d, case["dtype"], case["layout"])
        slots = torch.randperm(pages, generator=gen, device="cuda")[torch.arange(T, device="cuda") // P] * P
        slots = slots + torch.arange(T, device="cuda") % P
        if case["pad"]:
            slots[max(0, T - case["pad"]):] = -1
        s["slots"] = slots.to(torch.int32)
        return s
    ctx, new = _lens(case)
    kv = [c + m for c, m in zip(ctx, new)]
    counts = [_ceil(x, P) for x in kv]
    pages = sum(counts) + 2
    s["table"], _ = _table(gen, counts, max(counts), pages)
    s["kc"] = _cache(gen, pages, P, h_kv, d, case["dtype"], case["layout"])
    s["vc"] = _cache(gen, pages, P, h_kv, d, case["dtype"], case["layout"])
    T = sum(new)
    # twice the unit deviation: scores of a few units, so that the softmax has the weight on few keys
    s["q"] = (2 * torch.randn((T, case["h_q"], d), generator=gen, device="cuda")).to(dtype)
    s["o"] = torch.empty_like(s["q"])
    s["cu"] = _i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    s["kv"] = _i32(kv)
    s["host"] = (new, kv)
    s["scale"] = d ** -0.5
    s["max_kv"] = max(kv)
    if own:
        import linear_attention_serving_gdn_gb300 as gdn
        need = gdn.gdn_paged_attention_workspace_bytes(case["h_q"], h_kv, d, case["n"], T, max(kv))
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_maps(s):
    P = s["case"]["page"]
    table, F = s["table"], s["free"].shape[0]
    ctx, new = s["ctx"].long(), s["new"].long()
    n, width = table.shape
    have, total = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    need = total - have
    start = s["head"].long() + torch.cumsum(need, 0) - need
    ok = (total <= width) & ((need == 0) | (start + need <= F))
    col = torch.arange(width, device=table.device)
    fresh = ok[:, None] & (col >= have[:, None]) & (col < total[:, None])
    src = (start[:, None] + col - have[:, None]).clamp(0, F - 1)
    table.copy_(torch.where(fresh, s["free"][src], table))
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    kv = torch.where(ok, ctx + new, 0)
    head = s["head"] + torch.where(ok, need, 0).sum()
    t = torch.arange(s["slots"].shape[0], device=table.device)
    real = t < cu[-1]
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=n - 1)
    pos = ctx[r] + t - cu[r]
    live = real & ok[r]
    pos = torch.where(live, pos, 0)
    slots = torch.where(live, table[r, pos // P].long() * P + pos % P, -1)
    i32 = torch.int32
    return {"block_table": table, "cu_seqlens": cu.to(i32), "kv_lens": kv.to(i32), "slot_map": slots.to(i32),
            "positions": pos.to(i32), "free_head": head.to(i32)}


def _plain_write(s):
    P = s["case"]["page"]
    live = s["slots"] >= 0
    slots = s["slots"][live].long()
    s["kc"][slots // P, slots % P] = s["k"][live]
    s["vc"][slots // P, slots % P] = s["v"][live]
    return {"k_cache": s["kc"], "v_cache": s["vc"]}


def _plain_block(q, K, V, first_pos, window, scale, kv_len=None):
    """q [b][m][h_q][d], K/V [b][L][h_kv][d] in fp32; query u of row b stands at first_pos[b] + u."""
    b, m, h_q, d = q.shape
    L, h_kv = K.shape[1:3]
    g = h_q // h_kv
    qh = q.reshape(b, m, h_kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, h_kv, g * m, d)
    sc = torch.matmul(qh, K.permute(0, 2, 3, 1)).mul_(scale).view(b, h_kv, g, m, L)
    j = torch.arange(L, device=q.device)
    pos = first_pos[:, None] + torch.arange(m, device=q.device)
    dead = j > pos[..., None]
    if window:
        dead = dead | (j <= pos[..., None] - window)
    sc.masked_fill_(dead[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = sc.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, h_kv, g * m, L), V.transpose(1, 2)).view(b, h_kv, g, m, d)
    o = torch.where(l > 0, o / l, 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(b, m, h_q, d)


def _plain_attention(s):
    case, (new, kv) = s["case"], s["host"]
    q, table, P = s["q"], s["table"], case["page"]
    h_kv, d = case["h_kv"], case["d"]
    o = torch.empty_like(q)
    n, i, t = case["n"], 0, 0
    while i < n:
        # requests with as many new tokens go together, padded to the longest, while that stays small
        e, longest = i + 1, kv[i]
        while e < n and new[e] == new[i] and (e + 1 - i) * max(longest, kv[e]) * max(h_kv * d, case["h_q"] * new[i]) <= 1 << 29:
            longest = max(longest, kv[e])
            e += 1
        m = new[i]
        idx = table[i:e, :_ceil(longest, P)].long().clamp(min=0)
        K = s["kc"][idx].flatten(1, 2)[:, :longest].float()
        V = s["vc"][idx].flatten(1, 2)[:, :longest].float()
        first = (s["kv"][i:e] - m).long()
        Q = q[t:t + (e - i) * m].view(e - i, m, case["h_q"], d)
        # rows of a long chunk in blocks, so that the scores stay within a few GB
        step = max(1, (1 << 30) // ((e - i) * longest * case["h_q"]))
        for u in range(0, m, step):
            part = _plain_block(Q[:, u:u + step].float(), K, V, first + u, case["window"], s["scale"])
            o[t:t + (e - i) * m].view(e - i, m, case["h_q"], d)[:, u:u + step] = part.to(q.dtype)
        t += (e - i) * m
        i = e
    return o


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"maps": _plain_maps, "write": _plain_write, "attention": _plain_attention}[op](s)
    import linear_attention_serving_gdn_gb300 as gdn
    if op == "maps":
        gdn.gdn_paged_maps(s["ctx"], s["new"], s["table"], s["case"]["page"], s["num_pages"], s["cu"], s["kv"],
                           s["slots"], s["pos"], free_pages=s["free"], free_head=s["head"],
                           free_head_out=s["head_out"])
        return {"block_table": s["table"], "cu_seqlens": s["cu"], "kv_lens": s["kv"], "slot_map": s["slots"],
                "positions": s["pos"], "free_head": s["head_out"]}
    if op == "write":
        gdn.gdn_paged_kv_write(s["k"], s["v"], s["kc"], s["vc"], s["slots"])
        return {"k_cache": s["kc"], "v_cache": s["vc"]}
    gdn.gdn_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv"], s["o"], scale=s["scale"],
                            window=s["case"]["window"], max_kv_len=s["max_kv"], workspace=s["ws"])
    return s["o"]


def _pairs(new, kv, window):
    """(visible (query, key) pairs, K/V rows that some query sees) of one request."""
    ctx, pairs = kv - new, 0
    if not window:
        return new * ctx + new * (new + 1) // 2, kv
    for u in range(new):
        pairs += min(window, ctx + u + 1)
    return pairs, min(kv, window + new - 1)


def work(case):
    if case["op"] == "maps":
        ctx, new = _lens(case)
        P, n = case["page"], case["n"]
        fresh = sum(_ceil(c + m, P) - _ceil(c, P) for c, m in zip(ctx, new))
        seen = sum(1 for c in ctx if c % P)
        # lengths and table entries in; new entries (read from the free list), offsets, lengths, slots and positions out
        return {"bytes": 8 * n + 4 * seen + 8 * fresh + 4 * (n + 1) + 4 * n + 8 * (sum(new) + case["pad"]) + 8, "flops": 0}
    if case["op"] == "write":
        T = max(0, case["tokens"] - case["pad"])
        return {"bytes": 4 * case["tokens"] + 2 * 2 * 2 * T * case["h_kv"] * case["d"], "flops": 0}
    ctx, new = _lens(case)
    pairs = rows = 0
    for c, m in zip(ctx, new):
        p, r = _pairs(m, c + m, case["window"])
        pairs, rows = pairs + p, rows + r
    d = case["d"]
    return {"bytes": 2 * (2 * sum(new) * case["h_q"] * d + 2 * rows * case["h_kv"] * d),
            "flops": 4 * pairs * case["h_q"] * d}


def exact(case, seed):
    """Attention by its definition in 64 bits, one request and one K/V head at a time; the write by asking of each
    slot which token it holds; the maps have no computed numbers."""
    if case["op"] == "maps":
        return None
    s = prepare(case, seed)
    f64, P = torch.float64, case["page"]
    if case["op"] == "write":
        holds = torch.full((s["kc"].shape[0] * P,), -1, dtype=torch.long)
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                holds[slot] = t
        holds = holds.view(-1, P).cuda()
        out = {}
        for name, new, old in (("k_cache", s["k"], s["kc"]), ("v_cache", s["v"], s["vc"])):
            out[name] = torch.where((holds >= 0)[..., None, None], new[holds.clamp(min=0)].to(f64), old.to(f64))
        return out
    W = case["window"]
    groups = case["h_q"] // case["h_kv"]
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    bounds = s["cu"].tolist()
    for r, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        L = int(s["kv"][r])
        where = torch.arange(L, device="cuda")
        page, row = s["table"][r][where // P].long(), where % P
        for h in range(case["h_kv"]):
            K, V = s["kc"][page, row, h].to(f64), s["vc"][page, row, h].to(f64)
            for u0 in range(a, b, 512):
                u1 = min(b, u0 + 512)
                pos = L - b + torch.arange(u0, u1, device="cuda")[:, None]
                seen = where <= pos
                if W:
                    seen = seen & (where > pos - W)
                for g in range(groups):
                    score = s["q"][u0:u1, h * groups + g].to(f64) @ K.t() / case["d"] ** 0.5
                    score = torch.where(seen, score, -torch.inf)
                    out[u0:u1, h * groups + g] = torch.softmax(score, -1) @ V
    return out
