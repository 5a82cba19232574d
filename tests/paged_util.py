"""Inputs and 64-bit references of the paged-cache tests."""
from __future__ import annotations

import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def ceil(a, b):
    return -(-a // b)


def make_cache(gen, pages, page, h, d, dtype, layout):
    """K and V viewed as [pages][page][h][d] over one of three memory orders."""
    if layout == "nhd":
        k, v = (torch.randn((pages, page, h, d), generator=gen, device="cuda").to(dtype) for _ in range(2))
    elif layout == "hnd":
        k, v = (torch.randn((pages, h, page, d), generator=gen, device="cuda").to(dtype).permute(0, 2, 1, 3)
                for _ in range(2))
    else:  # "joint": K and V of a page side by side, rows padded by 8 elements
        kv = torch.randn((pages, 2, page, h, d + 8), generator=gen, device="cuda").to(dtype)
        k, v = kv[:, 0, ..., :d], kv[:, 1, ..., :d]
    return k, v


def make_case(lens, h_q, h_kv, d, dtype="bf16", page=16, layout="nhd", seed=0, pad=0, q_gain=2.0, extra_pages=3):
    """lens: (kv_len, new) per request.  Pages are a random permutation; unused table entries are -1."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[dtype]
    counts = [ceil(max(kv, 0), page) for kv, _ in lens]
    pages = sum(counts) + extra_pages
    k, v = make_cache(gen, pages, page, h_kv, d, dt, layout)
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(counts + [1]) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = perm[at:at + c]
        at += c
    new = [m for _, m in lens]
    T = sum(new) + pad
    # rows of q are slices of a wider projection output
    wide = torch.randn((T, h_q + 2 * h_kv, d), generator=gen, device="cuda") * q_gain
    q = wide.to(dt)[:, :h_q]
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    kv = torch.tensor([x for x, _ in lens], dtype=torch.int32, device="cuda")
    return {"q": q, "k": k, "v": v, "table": table, "cu": cu, "kv": kv, "lens": lens, "page": page,
            "unused": perm[at:]}


def run_attention(gdn, c, window=0, scale=None, max_kv_len=0, fill=float("nan"), stream=None):
    """One call; the workspace and the outputs start from a pattern that must not show."""
    T, h_q, d = c["q"].shape
    bound = max_kv_len or c["table"].shape[1] * c["page"]
    n = gdn.gdn_paged_attention_workspace_bytes(h_q, c["k"].shape[2], d, len(c["lens"]), T, bound)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full((T, h_q, d), fill, dtype=c["q"].dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    gdn.gdn_paged_attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], o, scale=scale, window=window,
                            max_kv_len=max_kv_len, workspace=ws, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    return o, int(st.item())


def reference(c, window=0, scale=None):
    """(o, tol) in 64 bits.  tol is the error that the documented roundings allow, element by element: half a step
    of the type for the output and for each weight (A = sum p |V| bounds the latter), and the fp32 product's error
    in a score (d roundings of its terms' absolute sum), which moves every weight by that factor both in the
    numerator and in the sum.  Weights under the smallest normal fp16 are off by half of its smallest step."""
    q, P = c["q"], c["page"]
    T, h_q, d = q.shape
    h_kv = c["k"].shape[2]
    scale = d ** -0.5 if scale is None else scale
    u = torch.finfo(q.dtype).eps / 2
    o = torch.zeros((T, h_q, d), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    t = 0
    for r, (kv, m) in enumerate(c["lens"]):
        if kv > 0 and m > 0:
            j = torch.arange(kv, device="cuda")
            page = c["table"][r, j // P].long()
            seen_page = (page >= 0) & (page < c["k"].shape[0])
            page = page.clamp(0, c["k"].shape[0] - 1)
            K, V = (torch.where(seen_page[:, None, None], x[page, j % P].double(), 0.0) for x in (c["k"], c["v"]))
            pos = kv - m + torch.arange(m, device="cuda")[:, None]
            vis = j <= pos
            if window:
                vis &= j > pos - window
            # rows that no query sees may hold anything
            dead = ~vis.any(0)
            K[dead], V[dead] = 0.0, 0.0
            for h in range(h_q):
                Q, Kh, Vh = q[t:t + m, h].double(), K[:, h * h_kv // h_q], V[:, h * h_kv // h_q]
                s = torch.where(vis, Q @ Kh.T * scale, -torch.inf)
                p = torch.where(vis.any(-1, keepdim=True), torch.softmax(s, -1), 0.0)  # no key: zeros
                terms = torch.where(vis, Q.abs() @ Kh.abs().T * scale, 0.0).amax(-1, keepdim=True)
                A = p @ Vh.abs()
                o[t:t + m, h] = p @ Vh
                tol[t:t + m, h] = (u * (o[t:t + m, h].abs() + A) * 1.02 + A * (2 * (d + 4) * terms * 2.0 ** -24 + 2.0 ** -18)
                                   + 2.0 ** -25 * (vis.double() @ Vh.abs() if q.dtype == torch.float16 else 0))
        t += m
    return o, tol


def assert_close(o, ref, tol, what=""):
    err = (o.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off; worst {err[bad].max().item():.3e} at "
                           f"{bad.nonzero()[0].tolist()} (allowed {tol[bad].min().item():.3e})")


def maps_reference(ctx, new, table, page, num_pages, capacity, free=None, head=0):
    """The rules of gdn_paged_maps one request after the other; table (list of lists) is changed in place."""
    width = len(table[0]) if table else 0
    cu, kv, slots, pos, status = [0], [], [-1] * capacity, [0] * capacity, 0
    served = head
    supply = head  # next entry of the list if every request so far had been served
    if free is not None and head < 0:
        status |= 4
        supply = len(free)
    tok = 0
    for i, (c, m) in enumerate(zip(ctx, new)):
        first, tok = tok, tok + max(m, 0)
        ok = not (c < 0 or m < 0 or c + m > 2 ** 31 - 1 or ceil(c + m, page) > width or tok > capacity)
        if not ok:
            status |= 4
        else:
            have = ceil(c, page)
            need = ceil(c + m, page) - have if free is not None else 0
            start, supply = supply, supply + need
            if need and start + need > len(free):
                ok = False
                status |= 8
            elif need:
                table[i][have:have + need] = free[start:start + need]
                served = start + need
        cu.append(min(tok, capacity))
        kv.append(c + m if ok else 0)
        if ok:
            for w in range(m):
                p = c + w
                page_id = table[i][p // page]
                good = 0 <= page_id < num_pages
                status |= 0 if good else 1
                slots[first + w] = page_id * page + p % page if good else -1
                pos[first + w] = p
    return cu, kv, slots, pos, served, status
