"""Serving steps of a hybrid block: a Gated DeltaNet layer, then a full-attention layer over a paged K/V cache.

The prompts run as one varlen step, then every decode step replays one CUDA graph: its lengths, pages and slots all
come from the device, so nothing is rebuilt on the host between tokens.

    python examples/hybrid_step.py [decode steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_serving_gdn_gb300 as gdn  # noqa: E402


class HybridBlock:
    """Random weights of one block, and the caches of up to ``max_reqs`` requests of ``max_len`` tokens."""

    def __init__(self, hidden=512, h_k=4, h_v=8, d_gdn=128, h_q=8, h_kv=2, d=128, page=64, max_reqs=8, max_len=4096,
                 seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=gen, device="cuda") * rows ** -0.5).bfloat16()

        self.hidden, self.page = hidden, page
        self.h_k, self.h_v, self.d_gdn = h_k, h_v, d_gdn
        self.h_q, self.h_kv, self.d = h_q, h_kv, d
        self.w_gdn = weight(hidden, (2 * h_k + h_v) * d_gdn + 2 * h_v)
        self.w_gdn_out = weight(h_v * d_gdn, hidden)
        self.w_qkv = weight(hidden, (h_q + 2 * h_kv) * d)
        self.w_out = weight(h_q * d, hidden)
        self.A_log = torch.zeros(h_v, device="cuda")
        self.dt_bias = torch.full((h_v,), -3.0, device="cuda")
        self.state = torch.zeros((max_reqs, h_v, d_gdn, d_gdn), device="cuda")
        self.width = -(-max_len // page)
        self.pages = max_reqs * self.width
        self.k_cache, self.v_cache = (torch.empty((self.pages, page, h_kv, d), dtype=torch.bfloat16, device="cuda")
                                      for _ in range(2))
        self.table = torch.full((max_reqs, self.width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(self.pages, generator=gen, device="cuda").to(torch.int32)
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers(self, n, tokens):
        """What a step of n requests and up to `tokens` tokens writes to."""
        i32 = dict(dtype=torch.int32, device="cuda")
        need = gdn.gdn_paged_attention_workspace_bytes(self.h_q, self.h_kv, self.d, n, tokens, self.width * self.page)
        return {"cu": torch.zeros(n + 1, **i32), "kv": torch.zeros(n, **i32), "slots": torch.zeros(tokens, **i32),
                "pos": torch.zeros(tokens, **i32), "ws": torch.empty(need, dtype=torch.uint8, device="cuda"),
                "rows": torch.arange(n, **i32)}

    def step(self, x, context, new, buf, cu_host=None):
        """One step over x [T][hidden]; `cu_host` (prompt lengths summed) for prompts, None for single tokens."""
        T, n = x.shape[0], new.shape[0]
        gdn.gdn_paged_maps(context, new, self.table[:n], self.page, self.pages, buf["cu"], buf["kv"], buf["slots"],
                           buf["pos"], free_pages=self.free, free_head=self.head, dev_status=self.status)
        # the Gated DeltaNet layer
        a, b = 2 * self.h_k * self.d_gdn, self.h_v * self.d_gdn
        y = x @ self.w_gdn
        q, k = (t.reshape(T, self.h_k, self.d_gdn).contiguous() for t in y[:, :a].chunk(2, 1))
        v = y[:, a:a + b].reshape(T, self.h_v, self.d_gdn).contiguous()
        ga, gb = (t.float().contiguous() for t in y[:, a + b:].chunk(2, 1))
        o = torch.empty_like(v)
        if cu_host is None:
            gdn.gdn_decode_packed_raw(q, k, v, ga, gb, self.A_log, self.dt_bias, self.state, buf["rows"], o,
                                      dev_status=self.status)
        else:
            qn, kn, g, beta = torch.empty_like(q), torch.empty_like(k), torch.empty_like(ga), torch.empty_like(gb)
            gdn.gdn_prep_inputs(q, k, ga, gb, self.A_log, self.dt_bias, qn, kn, g, beta)
            gdn.gdn_prefill_varlen(qn, kn, v, g, beta, buf["cu"], cu_host, o, state=self.state, dst_slot=buf["rows"],
                                   dev_status=self.status)
        x = x + o.reshape(T, -1) @ self.w_gdn_out
        # the full-attention layer
        qkv = (x @ self.w_qkv).view(T, -1, self.d)
        q, k, v = qkv.split([self.h_q, self.h_kv, self.h_kv], 1)
        gdn.gdn_paged_kv_write(k, v, self.k_cache, self.v_cache, buf["slots"], dev_status=self.status)
        o = torch.empty((T, self.h_q, self.d), dtype=x.dtype, device=x.device)
        gdn.gdn_paged_attention(q, self.k_cache, self.v_cache, self.table[:n], buf["cu"], buf["kv"], o,
                                workspace=buf["ws"], dev_status=self.status)
        return x + o.reshape(T, -1) @ self.w_out


def serve(block, prompts, steps, seed=1):
    """Prompts of the given lengths, then `steps` tokens of each: (prompt outputs, [decode outputs], inputs)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, total = len(prompts), sum(prompts)
    cu = [sum(prompts[:i]) for i in range(n + 1)]
    x = torch.randn((total, block.hidden), generator=gen, device="cuda").bfloat16()
    fed = torch.randn((steps, n, block.hidden), generator=gen, device="cuda").bfloat16()
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    first = block.step(x, torch.zeros_like(lens), lens, block.buffers(n, total), cu)
    # a decode step, captured: the context lengths move on inside the graph
    context, one, token = lens.clone(), torch.ones_like(lens), fed[0].clone()
    buf = block.buffers(n, n)
    saved = {k: getattr(block, k).clone() for k in ("state", "table", "head", "k_cache", "v_cache")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        block.step(token, context, one, buf)  # libraries settle before the capture
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        out = block.step(token, context, one, buf)
        context += 1
    for k, t in saved.items():
        getattr(block, k).copy_(t)
    outs = []
    for s in range(steps):
        token.copy_(fed[s])
        graph.replay()
        outs.append(out.clone())
    torch.cuda.synchronize()
    if block.status.item():
        raise gdn.GdnError(gdn.gdn_status_from_device(block.status.item()), "hybrid step")
    return first, outs, (x, fed, graph)


if __name__ == "__main__":
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    block = HybridBlock()
    prompts = [116, 321, 1059, 2000]
    _, outs, (_, _, graph) = serve(block, prompts, steps)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{len(prompts)} prompts, {steps} decode steps; {start.elapsed_time(end) / 20 * 1e3:.1f} us per replayed step")
