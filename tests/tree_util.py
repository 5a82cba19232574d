"""Inputs and 64-bit references of the tests over trees of drafted tokens."""
from __future__ import annotations

import random

import torch

from tests import paged_util as pu

SHAPES = ("mixed", "chain", "flat", "forest")


def parents_of(m, shape, seed=0):
    rng = random.Random(seed * 1009 + m)
    if shape == "chain":
        return list(range(-1, m - 1))
    if shape == "flat":
        return [-1] * m
    if shape == "forest":  # many roots, any earlier node
        return [rng.randint(-1, u - 1) if rng.random() < 0.7 else -1 for u in range(m)]
    return [int(u * rng.uniform(0.2, 0.8)) - 1 for u in range(m)]


def path_of(par, u):
    """Node u and those above it, from u on up."""
    out = []
    while u >= 0:
        out.append(u)
        u = par[u]
    return out


def words_of(trees):
    """int64 words of the trees' nodes."""
    words = [sum(1 << w for w in path_of(par, u) if w < 64) for par in trees for u in range(len(par))]
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")


def offsets(sizes):
    cu = [0]
    for m in sizes:
        cu.append(cu[-1] + m)
    return cu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- attention -------------------------------------------------------------------

def run_tree_attention(gdn, c, masks, scale=None, max_kv_len=0, fill=float("nan"), stream=None):
    """One call; the workspace and the outputs start from a pattern that must not show."""
    T, h_q, d = c["q"].shape
    bound = max_kv_len or c["table"].shape[1] * c["page"]
    n = gdn.gdn_paged_attention_workspace_bytes(h_q, c["k"].shape[2], d, len(c["lens"]), T, bound)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full((T, h_q, d), fill, dtype=c["q"].dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    gdn.gdn_tree_attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], masks, o, scale=scale,
                           max_kv_len=max_kv_len, workspace=ws, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    return o, int(st.item())


def attention_reference(c, masks, scale=None):
    """(o, tol) in 64 bits, node by node; the tolerance as in paged_util.reference (half a step for the output and each
    weight, the fp32 product's error in a score, fp16 weights under its smallest normal number)."""
    q, P = c["q"], c["page"]
    T, h_q, d = q.shape
    h_kv = c["k"].shape[2]
    scale = d ** -0.5 if scale is None else scale
    eps = torch.finfo(q.dtype).eps / 2
    o = torch.zeros((T, h_q, d), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    t = 0
    for r, (kv, m) in enumerate(c["lens"]):
        j = torch.arange(max(kv, 0), device="cuda")
        page = c["table"][r, j // P].long()
        good = (page >= 0) & (page < c["k"].shape[0])
        page = page.clamp(0, c["k"].shape[0] - 1)
        rows = [torch.where(good[:, None, None], x[page, j % P].double(), 0.0) for x in (c["k"], c["v"])]
        for u in range(m if kv > 0 else 0):
            word = int(masks[t + u]) & ((2 << u) - 1)
            sees = j < kv - m
            for w in range(u + 1):
                if word >> w & 1 and kv - m + w >= 0:
                    sees[kv - m + w] = True
            if not sees.any():
                continue
            K, V = (x[sees] for x in rows)
            for h in range(h_kv):
                heads = slice(h * h_q // h_kv, (h + 1) * h_q // h_kv)
                Q = q[t + u, heads].double()
                p = torch.softmax(Q @ K[:, h].T * scale, -1)
                terms = (Q.abs() @ K[:, h].abs().T * scale).amax(-1, keepdim=True)
                A, x = p @ V[:, h].abs(), p @ V[:, h]
                o[t + u, heads] = x
                tol[t + u, heads] = (eps * (x.abs() + A) * 1.02 + A * (2 * (d + 4) * terms * 2.0 ** -24 + 2.0 ** -18)
                                     + 2.0 ** -25 * (V[:, h].abs().sum(0) if q.dtype == torch.float16 else 0))
        t += m
    return o, tol


# ---- the gated delta rule ----------------------------------------------------------

def make_delta(trees, h_k, h_v, d, seed=0, pad=0, extra_slots=2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, sizes = len(trees), [len(p) for p in trees]
    T = sum(sizes) + pad

    def unit():
        x = torch.randn((T, h_k, d), generator=gen, device="cuda")
        return (x / x.norm(dim=-1, keepdim=True)).bfloat16()

    return {"trees": trees, "q": unit(), "k": unit(),
            "v": torch.randn((T, h_v, d), generator=gen, device="cuda").bfloat16(),
            "g": -0.3 * torch.rand((T, h_v), generator=gen, device="cuda"),
            "beta": torch.rand((T, h_v), generator=gen, device="cuda"),
            "state": 0.1 * torch.randn((n + extra_slots, h_v, d, d), generator=gen, device="cuda"),
            "slot": torch.randperm(n + extra_slots, generator=gen, device="cuda")[:n].to(torch.int32),
            "cu": i32(offsets(sizes)),
            "masks": torch.cat([words_of(trees), torch.zeros(pad, dtype=torch.int64, device="cuda")])}


def run_delta(gdn, c, max_nodes=64, scale=1.0, stream=None):
    o = torch.full_like(c["v"], float("nan"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    gdn.gdn_tree_decode(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], c["slot"], c["cu"], c["masks"], o,
                        max_nodes=max_nodes, dev_status=st, scale=scale, stream=stream)
    torch.cuda.synchronize()
    return o, int(st.item())


def delta_reference(c, scale=1.0):
    """(o, tol) in 64 bits: the recurrence from each node's parent.

    tol, element by element: half a step of bf16 for the output, and the documented errors of what is summed up,
    o = scale (G S^T q + sum_w C_w (v_w - G_w S^T k_w)): the state, C and the bracket each within 2^-15 (a sum of two
    bf16: 2^-8 of a rest under 2^-7), fp32 sums of d + 64 terms, decays as products of up to 64 exponentials (2^-22
    each); and C's own error, by the perturbation of the triangular system that it solves, C (I + A) = P:
    |dC| <= gamma (|P| + |C| |A|) |(I + A)^-1| with P and A from absolute values of the products."""
    h_v, d = c["v"].shape[1:]
    rep = h_v // c["q"].shape[1]
    o = torch.zeros(c["v"].shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    cu = c["cu"].tolist()
    fine = (d + 64) * 2.0 ** -23 + 64 * 2.0 ** -21
    for r, par in enumerate(c["trees"]):
        m, a = len(par), cu[r]
        if m == 0 or int(c["slot"][r]) < 0:
            continue
        q, k = (x[a:a + m].double().repeat_interleave(rep, 1) for x in (c["q"], c["k"]))
        v, alpha, beta = c["v"][a:a + m].double(), c["g"][a:a + m].double().exp(), c["beta"][a:a + m].double()
        S0 = c["state"][int(c["slot"][r])].double()
        states, G = [], []
        for u in range(m):
            S = (states[par[u]] if par[u] >= 0 else S0) * alpha[u][:, None, None]
            S = S + torch.einsum("hv,hk->hvk", beta[u][:, None] * (v[u] - torch.einsum("hvk,hk->hv", S, k[u])), k[u])
            states.append(S)
            G.append(alpha[u] * (G[par[u]] if par[u] >= 0 else 1.0))
            o[a + u] = scale * torch.einsum("hvk,hk->hv", S, q[u])
        G = torch.stack(G)
        E = torch.zeros((h_v, m, m), dtype=torch.float64, device="cuda")  # decays from node u to before w on its path
        on = torch.zeros((m, m), dtype=torch.float64, device="cuda")
        for u in range(m):
            run = torch.ones_like(alpha[0])
            for w in path_of(par, u):
                E[:, u, w], on[u, w] = run, 1.0
                run = run * alpha[w]
        bt = beta.T[:, None, :]
        kk, qk = torch.einsum("uhd,whd->huw", k, k), torch.einsum("uhd,whd->huw", q, k)
        kk_abs, qk_abs = torch.einsum("uhd,whd->huw", k.abs(), k.abs()), torch.einsum("uhd,whd->huw", q.abs(), k.abs())
        eye = torch.eye(m, dtype=torch.float64, device="cuda")
        inv = torch.linalg.inv(eye + E * bt * kk * (on - eye))
        C = (E * bt * qk) @ inv
        dC = fine * (E * bt * qk_abs + C.abs() @ (E * bt * kk_abs * (on - eye))) @ inv.abs()
        yabs = v.abs() + G[..., None] * torch.einsum("hvk,uhk->uhv", S0.abs(), k.abs())
        zabs = G[..., None] * torch.einsum("hvk,uhk->uhv", S0.abs(), q.abs())
        part = torch.einsum("huw,whv->uhv", C.abs(), yabs)
        tol[a:a + m] = (2.0 ** -8 * 1.01 * o[a:a + m].abs()
                        + scale * ((zabs + 3 * part) * (2.0 ** -15 + fine) + torch.einsum("huw,whv->uhv", dC, yabs)))
    return o, tol


assert_close = pu.assert_close
