"""Speculative decoding in trees through a hybrid block: a Gated DeltaNet layer, then a full-attention layer with rotary
positions over a paged K/V cache.

The prompts run as one varlen step.  Then each step verifies a tree of drafted tokens per request in one pass, from the
requests' states and caches, which it leaves as they are (the nodes' keys and values lie behind the context); what is
accepted, a path from a root, is committed to both.

    python examples/tree_step.py [nodes per tree]
"""
from __future__ import annotations

import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from hybrid_step import HybridBlock, gdn  # noqa: E402


def draft(nodes, seed):
    """A tree's parents, as a drafter grows it: numbers below the node's own, -1 for a child of the last cached token."""
    rng = random.Random(seed)
    return [int(u * rng.uniform(0.2, 0.8)) - 1 for u in range(nodes)]


class TreeBlock(HybridBlock):
    """The block with rotary positions on the first ``rotary`` elements of its attention heads."""

    def __init__(self, rotary=64, **kw):
        super().__init__(**kw)
        self.freq = gdn.gdn_rotary_frequencies(rotary, 1000000.0, "yarn", 4.0, original_length=32768).cuda()

    def buffers(self, n, tokens):
        return {**super().buffers(n, tokens), "masks": torch.zeros(tokens, dtype=torch.int64, device="cuda")}

    def step(self, x, context, new, buf, cu_host=None, parents=None):
        """One step over x [T][hidden]: prompts (`cu_host`: their lengths summed) or trees (`parents` [T]).  Gives the
        outputs, and of trees what a commit needs."""
        T, n = x.shape[0], new.shape[0]
        gdn.gdn_paged_maps(context, new, self.table[:n], self.page, self.pages, buf["cu"], buf["kv"], buf["slots"],
                           buf["pos"], free_pages=self.free, free_head=self.head, dev_status=self.status)
        if parents is not None:
            gdn.gdn_tree_maps(parents, buf["cu"], buf["kv"], buf["masks"], buf["pos"], dev_status=self.status)
        # the Gated DeltaNet layer
        a, b = 2 * self.h_k * self.d_gdn, self.h_v * self.d_gdn
        y = x @ self.w_gdn
        q, k = (t.reshape(T, self.h_k, self.d_gdn).contiguous() for t in y[:, :a].chunk(2, 1))
        v = y[:, a:a + b].reshape(T, self.h_v, self.d_gdn).contiguous()
        g, beta = (t.float().contiguous() for t in y[:, a + b:].chunk(2, 1))
        gdn.gdn_prep_inputs(q, k, g, beta, self.A_log, self.dt_bias, q, k, g, beta)
        o = torch.empty_like(v)
        if parents is None:
            gdn.gdn_prefill_varlen(q, k, v, g, beta, buf["cu"], cu_host, o, state=self.state, dst_slot=buf["rows"],
                                   dev_status=self.status)
        else:
            gdn.gdn_tree_decode(q, k, v, g, beta, self.state, buf["rows"], buf["cu"], buf["masks"], o,
                                dev_status=self.status)
        kept = (q, k, v, g, beta)
        x = x + o.reshape(T, -1) @ self.w_gdn_out
        # the full-attention layer
        qkv = (x @ self.w_qkv).view(T, -1, self.d)
        q, k, v = qkv.split([self.h_q, self.h_kv, self.h_kv], 1)
        gdn.gdn_rotary(q, k, buf["pos"], self.freq)
        gdn.gdn_paged_kv_write(k, v, self.k_cache, self.v_cache, buf["slots"], dev_status=self.status)
        o = torch.empty((T, self.h_q, self.d), dtype=x.dtype, device=x.device)
        if parents is None:
            gdn.gdn_paged_attention(q, self.k_cache, self.v_cache, self.table[:n], buf["cu"], buf["kv"], o,
                                    workspace=buf["ws"], dev_status=self.status)
        else:
            gdn.gdn_tree_attention(q, self.k_cache, self.v_cache, self.table[:n], buf["cu"], buf["kv"], buf["masks"], o,
                                   workspace=buf["ws"], dev_status=self.status)
        return x + o.reshape(T, -1) @ self.w_out, kept

    def commit(self, kept, buf, path, context):
        """Accepts path [n][L] of node numbers, -1 behind its end: the states go on over it, its keys and values move up
        behind the context, which grows by it."""
        L = path.shape[1]
        if L == 0 or kept[0].shape[0] == 0:
            return
        live, cu = path >= 0, buf["cu"][:-1].long()[:, None]
        # (behind a path's end token 0, which is always there: a request may have no nodes)
        tok = torch.where(live, cu + path, 0).flatten()
        # (zeros throughout: with g = beta = 0 the state stays as it is, but for 0 times a k or v that is not finite)
        q, k, v, g, beta = (t[tok].masked_fill_(~live.flatten().view(-1, *[1] * (t.dim() - 1)), 0.0) for t in kept)
        gdn.gdn_decode_multi(L, q, k, v, g, beta, self.state, buf["rows"], torch.empty_like(v), dev_status=self.status)
        place = torch.where(live, cu + torch.arange(L, device=path.device), 0)
        to = torch.where(live, buf["slots"][place], -1).flatten()  # (not written behind a path's end)
        slots = buf["slots"][tok].long()
        k, v = (c[slots // self.page, slots % self.page] for c in (self.k_cache, self.v_cache))
        gdn.gdn_paged_kv_write(k, v, self.k_cache, self.v_cache, to, dev_status=self.status)
        context += live.sum(1).to(context.dtype)

    def give_back(self, context, n):
        """Pages behind the contexts return to the free list (a serving loop does so with its own bookkeeping)."""
        keep = torch.arange(self.width, device="cuda") < ((context.long() + self.page - 1) // self.page)[:, None]
        spare = self.table[:n][~keep & (self.table[:n] >= 0)]
        self.head -= spare.numel()
        self.free[int(self.head):int(self.head) + spare.numel()] = spare
        self.table[:n][~keep] = -1


def check(block):
    torch.cuda.synchronize()
    if block.status.item():
        raise gdn.GdnError(gdn.gdn_status_from_device(block.status.item()), "tree step")


if __name__ == "__main__":
    nodes = int(sys.argv[1]) if len(sys.argv) > 1 else 32
    block = TreeBlock()
    prompts = [116, 321, 1059, 2000]
    n, gen = len(prompts), torch.Generator(device="cuda").manual_seed(1)
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    context = torch.zeros_like(lens)
    x = torch.randn((sum(prompts), block.hidden), generator=gen, device="cuda").bfloat16()
    block.step(x, context, lens, block.buffers(n, sum(prompts)), [sum(prompts[:i]) for i in range(n + 1)])
    context += lens
    trees = [draft(nodes, s) for s in range(n)]
    parents = torch.tensor(sum(trees, []), dtype=torch.int32, device="cuda")
    new = torch.full((n,), nodes, dtype=torch.int32, device="cuda")
    x = torch.randn((n * nodes, block.hidden), generator=gen, device="cuda").bfloat16()
    buf = block.buffers(n, n * nodes)
    block.step(x, context, new, buf, parents=parents)  # takes the pages
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(x, context, new, buf, parents=parents)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    check(block)
    print(f"{n} trees of {nodes} nodes; {start.elapsed_time(end) / 20 * 1e3:.1f} us per replayed verification")
