"""Cases of the operators that verify a tree of drafted tokens in a hybrid decoder: the tree's maps, rotary positions,
attention of a tree over the paged cache, and the gated delta rule along a tree.

``run`` computes an operator in its plain form (elementary torch operations) or, with ``own`` set, through the
framework's entry points.  A case is a plain dict; ``prepare`` turns it into the tensors a serving program holds
before the step.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# Tree sizes and shapes and the contexts' lengths are derived from the case's own "lens_seed", so that `work` and
# `prepare` agree on them; the values of the tensors come from the seed given to `prepare`.

def _maps(name, n, nodes_lo, nodes_hi, ctx_lo, ctx_hi, shape="mixed", pad=0, lens_seed=0):
    """n requests, each a tree of nodes_lo..nodes_hi drafted tokens behind ctx_lo..ctx_hi cached ones."""
    return {"name": name, "op": "maps", "n": n, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "shape": shape, "pad": pad, "lens_seed": lens_seed}


def _rotary(name, tokens, h_q, h_kv, d, rot, dtype, interleaved, max_pos, scaling="none", factor=1.0):
    """q and k of one projection's output, `rot` elements of each head turned by positions up to max_pos."""
    return {"name": name, "op": "rotary", "tokens": tokens, "h_q": h_q, "h_kv": h_kv, "d": d, "rot": rot,
            "dtype": dtype, "interleaved": interleaved, "max_pos": max_pos, "scaling": scaling, "factor": factor}


def _attn(name, n, nodes_lo, nodes_hi, ctx_lo, ctx_hi, h_q, h_kv, d, dtype, page, layout="nhd", shape="mixed",
          lens_seed=0):
    return {"name": name, "op": "attention", "n": n, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "h_q": h_q, "h_kv": h_kv, "d": d, "dtype": dtype, "page": page, "layout": layout,
            "shape": shape, "lens_seed": lens_seed}


def _delta(name, n, nodes_lo, nodes_hi, h_k, h_v, d, shape="mixed", lens_seed=0):
    return {"name": name, "op": "delta", "n": n, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "ctx_lo": 0, "ctx_hi": 0,
            "h_k": h_k, "h_v": h_v, "d": d, "shape": shape, "lens_seed": lens_seed}


def listed():
    return [
        # the trees of a small batch: five to sixteen drafted tokens each, padded to the captured graph's size
        _maps("maps_8_trees", 8, 5, 16, 100, 4000, pad=20),
        # a large batch, single tokens and trees of up to 64
        _maps("maps_512_trees", 512, 1, 64, 0, 20000, lens_seed=1),
        # eight decode rows, a quarter of each head turned
        _rotary("rotary_decode_8", 8, 16, 2, 256, 64, "bf16", False, 4000),
        # 256 trees of 16 drafted tokens far behind the trained length, pairs next to each other
        _rotary("rotary_trees_4096", 4096, 16, 2, 256, 64, "fp16", True, 1000000, "yarn", 32.0),
        # a long prompt chunk, whole heads
        _rotary("rotary_chunk_32768", 32768, 32, 8, 128, 128, "bf16", False, 131072),
        # one user's tree of seven drafted tokens: nothing but latency
        _attn("attn_one_tree", 1, 7, 7, 1058, 1058, 16, 2, 256, "bf16", 64),
        # 64 users' trees of up to 64 tokens on 1088-token blocks
        _attn("attn_64_trees", 64, 16, 64, 500, 8000, 16, 2, 256, "bf16", 1088, lens_seed=2),
        # few very long contexts, small pages
        _attn("attn_long", 8, 25, 32, 60000, 100000, 32, 8, 128, "fp16", 16, layout="hnd", lens_seed=3),
        # small trees and rows without a draft, one K/V head per query head
        _attn("attn_small_trees", 128, 1, 12, 2000, 8000, 16, 16, 64, "bf16", 32, lens_seed=4),
        # one user's tree in a linear-attention layer
        _delta("delta_one_tree", 1, 12, 12, 16, 16, 128),
        # 256 users' small trees
        _delta("delta_256_trees", 256, 4, 12, 16, 16, 128, lens_seed=5),
        # 64 users' trees of up to 64 tokens, two value heads per key head
        _delta("delta_64_trees", 64, 33, 64, 16, 32, 128, lens_seed=6),
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm of lo..hi, odd values included."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random())) + rng.randint(0, 1)))


def draw(rng: random.Random):
    op = rng.choice(["maps", "rotary", "rotary", "attention", "attention", "attention", "delta", "delta"])
    seed = rng.randrange(1 << 30)
    shape = rng.choice(["mixed", "mixed", "mixed", "chain", "flat"])
    if op == "rotary":
        h_q, h_kv, d, rot = rng.choice([(16, 2, 256, 64), (16, 2, 256, 256), (32, 8, 128, 128), (16, 16, 64, 64),
                                        (12, 4, 64, 32), (20, 4, 128, 64), (32, 8, 128, 96), (5, 1, 80, 20)])
        tokens = _log_int(rng, 1, 32768 * 5120 // ((h_q + h_kv) * d))
        scaling, factor = rng.choice([("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0), ("yarn", 40.0)])
        return _rotary("", tokens, h_q, h_kv, d, rot, rng.choice(["bf16", "fp16"]), rng.random() < 0.5,
                       _log_int(rng, 100, 2000000), scaling, factor)
    hi = _log_int(rng, 1, 64)
    lo = rng.randint(1, hi)
    if op == "maps":
        return _maps("", _log_int(rng, 1, 512), lo, hi, 0, _log_int(rng, 64, 20000), shape,
                     pad=rng.choice([0, rng.randint(1, 64)]), lens_seed=seed)
    if op == "delta":
        h_k, h_v, d = rng.choice([(16, 16, 128), (16, 32, 128), (4, 8, 128), (8, 8, 64), (4, 12, 64)])
        # states and tokens within the largest listed case's
        n = _log_int(rng, 1, min(256, 64 * 32 * 128 * 128 // (h_v * d * d)))
        return _delta("", n, lo, hi, h_k, h_v, d, shape, seed)
    h_kv, group, d = rng.choice([(2, 8, 256), (4, 4, 256), (8, 4, 128), (4, 8, 128), (4, 5, 128), (16, 1, 128),
                                 (16, 1, 64), (4, 3, 64), (1, 16, 64)])
    ctx = _log_int(rng, 16, 100000)
    # products and cache within the largest listed case's
    most = min((1 << 30) // (ctx * h_kv * d), 8 * 28 * 80000 * 32 * 128 // (ctx * hi * h_kv * group * d))
    n = _log_int(rng, 1, max(1, min(256, most)))
    return _attn("", n, lo, hi, rng.randint(0, ctx), ctx, h_kv * group, h_kv, d, rng.choice(["bf16", "fp16"]),
                 rng.choice([16, 32, 48, 64, 128, 1088]), rng.choice(["nhd", "hnd"]), shape, seed)


def _trees(case):
    """Host lists: each request's context length, and its nodes' parents (indices in the request; -1: the last
    cached token)."""
    rng = random.Random(case["lens_seed"] * 1000003 + case["n"])
    out = []
    for _ in range(case["n"]):
        ctx, m = rng.randint(case["ctx_lo"], case["ctx_hi"]), rng.randint(case["nodes_lo"], case["nodes_hi"])
        if case["shape"] == "chain":
            par = list(range(-1, m - 1))
        elif case["shape"] == "flat":
            par = [-1] * m
        else:  # as drafts are grown: several children per node, six to nine levels at 64 nodes
            par = [int(u * rng.uniform(0.2, 0.8)) - 1 for u in range(m)]
        out.append((ctx, par))
    return out


def _depths(par):
    depth = []
    for p in par:
        depth.append(1 + (depth[p] if p >= 0 else 0))
    return depth


def _ceil(a, b):
    return -(-a // b)


def _inverse_frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    rot, base, factor = case["rot"], 10000.0, case["factor"]
    if case["scaling"] == "ntk":
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        f = [x / factor for x in f]
    if case["scaling"] == "yarn":  # pairs that turn often keep their speed, those that turn less than once are stretched
        def pair(turns):
            return rot * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        f = [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)]
    return f


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(gen, pages, page, h, d, dtype, layout):
    """A K or V cache viewed as [pages][page][h][d]; the "hnd" layout holds its pages head by head."""
    shape = (pages, page, h, d) if layout == "nhd" else (pages, h, page, d)
    t = torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[dtype])
    return t if layout == "nhd" else t.permute(0, 2, 1, 3)


def _masks(trees):
    """One 64-bit word per node: bit v is set where node v is the node itself or above it."""
    out = []
    for _, par in trees:
        own_words = []
        for u, p in enumerate(par):
            own_words.append((1 << u) | (own_words[p] if p >= 0 else 0))
        out += [w - (1 << 64) if w >> 63 else w for w in own_words]
    return torch.tensor(out, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rotary":
        T, h_q, h_kv, d = case["tokens"], case["h_q"], case["h_kv"], case["d"]
        qkv = torch.randn((T, h_q + 2 * h_kv, d), generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        s["q"], s["k"] = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv]
        s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=gen, device="cuda", dtype=torch.int32)
        s["q_out"], s["k_out"] = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (s["q"], s["k"]))
        s["magnitude"] = _magnitude(case)
        if own:
            import linear_attention_serving_gdn_gb300 as gdn
            s["freq"] = gdn.gdn_rotary_frequencies(case["rot"], 10000.0, case["scaling"], case["factor"],
                                                   original_length=32768).cuda()
        else:
            s["freq"] = torch.tensor(_inverse_frequencies(case), dtype=torch.float64, device="cuda")
        return s
    trees = _trees(case)
    sizes = [len(par) for _, par in trees]
    T, n = sum(sizes), case["n"]
    cu = [0]
    for m in sizes:
        cu.append(cu[-1] + m)
    s["cu"] = _i32(cu)
    if case["op"] == "maps":
        shift = random.Random(seed).randrange(64)  # other seeds are other steps: the contexts move on
        s["kv"] = _i32([ctx + shift + m for (ctx, _), m in zip(trees, sizes)])
        s["parents"] = _i32(sum((par for _, par in trees), []) + [-1] * case["pad"])
        s["masks"] = torch.zeros(T + case["pad"], dtype=torch.int64, device="cuda")
        s["pos"] = torch.zeros(T + case["pad"], dtype=torch.int32, device="cuda")
        return s
    s["masks"] = _masks(trees)
    s["sizes"] = sizes
    if case["op"] == "attention":
        P, h_q, h_kv, d = case["page"], case["h_q"], case["h_kv"], case["d"]
        kv = [ctx + m for (ctx, _), m in zip(trees, sizes)]
        counts = [_ceil(x, P) for x in kv]
        pages, width = sum(counts) + 2, max(counts)
        perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        cnt = torch.tensor(counts, device="cuda")
        first, col = torch.cumsum(cnt, 0) - cnt, torch.arange(width, device="cuda")
        s["table"] = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        live = col[None, :] < cnt[:, None]
        s["table"][live] = perm[(first[:, None] + col[None, :])[live]]
        s["kc"] = _cache(gen, pages, P, h_kv, d, case["dtype"], case["layout"])
        s["vc"] = _cache(gen, pages, P, h_kv, d, case["dtype"], case["layout"])
        # twice the unit deviation: scores of a few units, so that the softmax has the weight on few keys
        s["q"] = (2 * torch.randn((T, h_q, d), generator=gen, device="cuda")).to(DTYPES[case["dtype"]])
        s["o"] = torch.empty_like(s["q"])
        s["kv"], s["kv_host"], s["scale"] = _i32(kv), kv, d ** -0.5
        if own:
            import linear_attention_serving_gdn_gb300 as gdn
            need = gdn.gdn_paged_attention_workspace_bytes(h_q, h_kv, d, n, T, max(kv))
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return s
    # the gated delta rule: unit keys and queries, decays near one, states as a long context leaves them
    h_k, h_v, d = case["h_k"], case["h_v"], case["d"]
    q, k = (torch.randn((T, h_k, d), generator=gen, device="cuda") for _ in range(2))
    s["q"], s["k"] = ((x / x.norm(dim=-1, keepdim=True)).bfloat16() for x in (q, k))
    s["v"] = torch.randn((T, h_v, d), generator=gen, device="cuda").bfloat16()
    s["g"] = -0.3 * torch.rand((T, h_v), generator=gen, device="cuda")
    s["beta"] = torch.rand((T, h_v), generator=gen, device="cuda")
    s["state"] = 0.1 * torch.randn((n + 3, h_v, d, d), generator=gen, device="cuda")
    s["slot"] = torch.randperm(n + 3, generator=gen, device="cuda")[:n].to(torch.int32)
    s["o"] = torch.empty_like(s["v"])
    # each node's parent, padded to the largest tree: what the plain form walks
    most = max(sizes)
    s["parent"] = torch.tensor([[par[u] if u < len(par) else -1 for _, par in trees] for u in range(most)], device="cuda")
    s["token"] = torch.tensor([[a + min(u, m - 1) for a, m in zip(cu, sizes)] for u in range(most)], device="cuda")
    s["live"] = torch.tensor([[u < m for m in sizes] for u in range(most)], device="cuda")
    s["most"] = most
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_maps(s):
    cu, kv, parents = s["cu"].long(), s["kv"].long(), s["parents"].long()
    T = parents.numel()
    t = torch.arange(T, device=parents.device)
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=kv.numel() - 1)
    live = t < cu[-1]
    u = t - cu[r]
    mask = torch.where(live, torch.ones_like(u) << u.clamp(0, 63), 0)
    up = torch.where(live & (parents >= 0), cu[r] + parents, -1)  # pointers are doubled: 2, 4, ... levels up
    for _ in range(6):
        mask = torch.where(up >= 0, mask | mask[up.clamp(min=0)], mask)
        up = torch.where(up >= 0, up[up.clamp(min=0)], -1)
    depth = sum((mask >> b) & 1 for b in range(64))
    pos = torch.where(live, kv[r] - (cu[r + 1] - cu[r]) + depth - 1, 0)
    return {"masks": mask, "positions": pos.to(torch.int32)}


def _plain_rotary(s):
    case = s["case"]
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        turned, rest = x[..., :case["rot"]], x[..., case["rot"]:]
        if case["interleaved"]:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = turned.chunk(2, -1)
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out[name] = torch.cat([turned, rest], -1).to(s[name].dtype)
    return out


def _plain_attention(s):
    case, P = s["case"], s["case"]["page"]
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    o = torch.empty_like(s["q"])
    t = 0
    for i, (m, kv) in enumerate(zip(s["sizes"], s["kv_host"])):
        idx = s["table"][i, :_ceil(kv, P)].long()
        K = s["kc"][idx].flatten(0, 1)[:kv].float()
        V = s["vc"][idx].flatten(0, 1)[:kv].float()
        q = s["q"][t:t + m].float().view(m, h_kv, h_q // h_kv, d).permute(1, 2, 0, 3).reshape(h_kv, -1, d)
        sc = torch.matmul(q, K.permute(1, 2, 0)).mul_(s["scale"]).view(h_kv, -1, m, kv)
        word = s["masks"][t:t + m]
        sees = (word[:, None] >> torch.arange(m, device=word.device)) & 1
        sc[..., kv - m:].masked_fill_(sees == 0, float("-inf"))
        p = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
        x = torch.matmul(p.view(h_kv, -1, kv), V.transpose(0, 1)).view(h_kv, -1, m, d) / p.sum(-1, keepdim=True)
        o[t:t + m] = x.permute(2, 0, 1, 3).reshape(m, h_q, d).to(o.dtype)
        t += m
    return o


def _plain_delta(s):
    """The recurrence, node after node over all requests at once; every node's state is kept for its children."""
    case = s["case"]
    n, rep, d, h_v = case["n"], case["h_v"] // case["h_k"], case["d"], case["h_v"]
    states = torch.empty((s["most"] + 1, n, h_v, d, d), dtype=torch.float32, device="cuda")  # [d_v][d_k]; the last: entering
    states[-1] = s["state"][s["slot"].long()]
    rows = torch.arange(n, device="cuda")
    o = torch.empty_like(s["o"])
    for u in range(s["most"]):
        t = s["token"][u]
        q, k = (x[t].float().repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
        S = states[s["parent"][u], rows] * s["g"][t].exp()[..., None, None]
        fresh = s["beta"][t][..., None] * (s["v"][t].float() - torch.matmul(S, k[..., None])[..., 0])
        S = S + fresh[..., None] * k[..., None, :]
        states[u] = S
        live = s["live"][u]
        o[t[live]] = torch.matmul(S, q[..., None])[..., 0][live].to(o.dtype)
    return o


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"maps": _plain_maps, "rotary": _plain_rotary, "attention": _plain_attention, "delta": _plain_delta}[op](s)
    import linear_attention_serving_gdn_gb300 as gdn
    if op == "maps":
        gdn.gdn_tree_maps(s["parents"], s["cu"], s["kv"], s["masks"], s["pos"])
        return {"masks": s["masks"], "positions": s["pos"]}
    if op == "rotary":
        gdn.gdn_rotary(s["q"], s["k"], s["pos"], s["freq"], s["q_out"], s["k_out"],
                       interleaved=s["case"]["interleaved"], magnitude=s["magnitude"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "attention":
        gdn.gdn_tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv"], s["masks"], s["o"],
                               scale=s["scale"], max_kv_len=max(s["kv_host"]), workspace=s["ws"])
        return s["o"]
    gdn.gdn_tree_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["slot"], s["cu"], s["masks"], s["o"],
                        max_nodes=s["most"])
    return s["o"]


def work(case):
    if case["op"] == "rotary":
        row, T = (case["h_q"] + case["h_kv"]) * case["d"], case["tokens"]
        pairs = T * (case["h_q"] + case["h_kv"]) * case["rot"] // 2
        return {"bytes": 2 * 2 * row * T + 4 * T, "flops": 6 * pairs}
    trees = _trees(case)
    T, n = sum(len(par) for _, par in trees), case["n"]
    if case["op"] == "maps":
        T += case["pad"]
        return {"bytes": 4 * T + 4 * (n + 1) + 4 * n + 12 * T, "flops": 0}
    seen = sum(sum(_depths(par)) for _, par in trees)  # (node, node at or above it) pairs
    if case["op"] == "attention":
        pairs = seen + sum(ctx * len(par) for ctx, par in trees)
        keys, d = sum(ctx + len(par) for ctx, par in trees), case["d"]
        return {"bytes": 2 * (2 * T * case["h_q"] * d + 2 * keys * case["h_kv"] * d) + 8 * T,
                "flops": 4 * pairs * case["h_q"] * d}
    h_k, h_v, d = case["h_k"], case["h_v"], case["d"]
    # states, q, k, v, o, gates and words; each node's two products with the entering state, and three dot products or
    # sums of d terms per pair (k.k, q.k, the update's part in the output)
    return {"bytes": 4 * n * h_v * d * d + 2 * T * 2 * (h_k + h_v) * d + 8 * T * h_v + 8 * T + 4 * n,
            "flops": h_v * (4 * T * d * d + 6 * seen * d)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """Rotary: the pair as a complex number times magnitude * exp(i angle).  Attention: each request's softmax over the
    context and the nodes at or above the query.  Delta rule: o = q^T S walked from the node to the root, q^T S_u =
    c v_u + p^T S_parent with c = beta (q.k), p = alpha (q - c k).  The maps are whole numbers."""
    f64 = torch.float64
    if case["op"] == "maps":
        return None
    s = prepare(case, seed)
    if case["op"] == "rotary":
        freq = torch.tensor(_inverse_frequencies(case), dtype=f64, device="cuda")
        turn = torch.polar(torch.full_like(freq, _magnitude(case)), s["pos"].to(f64)[:, None] * freq)[:, None]
        out = {}
        for name in ("q", "k"):
            x, rot = s[name].to(f64).clone(), case["rot"]
            at = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(x[..., at[0]], x[..., at[1]]) * turn
            x[..., at[0]], x[..., at[1]] = z.real, z.imag
            out[name] = x
        return out
    trees, bounds = _trees(case), s["cu"].tolist()
    if case["op"] == "attention":
        P, groups = case["page"], case["h_q"] // case["h_kv"]
        out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
        for r, (ctx, par) in enumerate(trees):
            a, m = bounds[r], len(par)
            sees = torch.zeros((m, ctx + m), dtype=torch.bool)
            sees[:, :ctx] = True
            for u, p in enumerate(par):
                if p >= 0:
                    sees[u] = sees[p]
                sees[u, ctx + u] = True
            where, sees = torch.arange(ctx + m, device="cuda"), sees.cuda()
            page, row = s["table"][r][where // P].long(), where % P
            for h in range(case["h_kv"]):
                K, V = s["kc"][page, row, h].to(f64), s["vc"][page, row, h].to(f64)
                heads = slice(h * groups, (h + 1) * groups)
                score = torch.einsum("ugd,jd->ugj", s["q"][a:a + m, heads].to(f64), K) / case["d"] ** 0.5
                score = torch.where(sees[:, None], score, -torch.inf)
                out[a:a + m, heads] = torch.einsum("ugj,jd->ugd", torch.softmax(score, -1), V)
        return out
    rep = case["h_v"] // case["h_k"]
    out = torch.zeros(s["o"].shape, dtype=f64, device="cuda")
    for r, (_, par) in enumerate(trees):
        a, m = bounds[r], len(par)
        q, k = (x[a:a + m].to(f64).repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
        v, alpha, beta = s["v"][a:a + m].to(f64), s["g"][a:a + m].to(f64).exp(), s["beta"][a:a + m].to(f64)
        S0 = s["state"][s["slot"][r].long()].to(f64)
        p, o, at = q.clone(), torch.zeros_like(v), torch.arange(m, device="cuda")
        above = torch.tensor(par + [-1], device="cuda")
        while bool((at >= 0).any()):
            i = torch.nonzero(at >= 0)[:, 0]
            w = at[i]
            c = beta[w] * (p[i] * k[w]).sum(-1)
            o[i] += c[..., None] * v[w]
            p[i] = alpha[w][..., None] * (p[i] - c[..., None] * k[w])
            at = torch.where(at >= 0, above[at], -1)
        out[a:a + m] = o + torch.einsum("uhk,hvk->uhv", p, S0)
    return out
