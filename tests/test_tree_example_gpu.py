"""The example's verification of trees: every node against its path as part of the prompt, before and after a commit."""
import importlib.util
import os

import pytest
import torch

from tests import tree_util as tu

pytestmark = pytest.mark.gpu


def load_example():
    folder = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")
    spec = importlib.util.spec_from_file_location("tree_step", os.path.join(folder, "tree_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def prompts_of(ex, x, lens):
    """Whole sequences through a fresh block: outputs of all tokens."""
    block = ex.TreeBlock(max_reqs=len(lens))
    cu = tu.offsets(lens)
    out, _ = block.step(x, tu.i32([0] * len(lens)), tu.i32(lens), block.buffers(len(lens), cu[-1]), cu)
    ex.check(block)
    return block, out


def verified_against_prompts(ex, outs, x, trees, before):
    """Each node's output against the last of the sequence of what its request has seen (`before`) and its path."""
    cu = tu.offsets([len(p) for p in trees])
    seqs, at = [], []
    for r, par in enumerate(trees):
        for u in range(0, len(par), 3):
            path = tu.path_of(par, u)[::-1]
            seqs.append(torch.cat([before[r], x[cu[r] + torch.tensor(path, device="cuda")]]))
            at.append(cu[r] + u)
    lens = [len(s) for s in seqs]
    _, want = prompts_of(ex, torch.cat(seqs), lens)
    ends = torch.tensor(tu.offsets(lens)[1:], device="cuda") - 1
    for t, w in zip(at, want[ends].float()):
        # the recurrence in one form against the other and bf16 in between: 2e-2 of the values' size each, as the two
        # layers are held to by themselves
        assert (outs[t].float() - w).abs().max() <= 4e-2 * (1 + w.abs().max()), t


def test_nodes_match_their_paths_as_prompts():
    ex = load_example()
    prompts, sizes = [116, 63, 7], [14, 31, 5]
    n, gen = len(prompts), torch.Generator(device="cuda").manual_seed(3)

    def tokens(T, hidden):
        return torch.randn((T, hidden), generator=gen, device="cuda").bfloat16()

    x0 = tokens(sum(prompts), 512)
    block, _ = prompts_of(ex, x0, prompts)
    context = tu.i32(prompts)
    before = list(x0.split(prompts))
    for round_, paths in enumerate(([0, 1, 2], [3, 0, 1])):  # accepted lengths
        trees = [ex.draft(m, 10 * round_ + r) for r, m in enumerate(sizes)]
        x = tokens(sum(sizes), 512)
        buf = block.buffers(n, sum(sizes))
        parents, new = tu.i32(sum(trees, [])), tu.i32(sizes)
        state = block.state.clone()
        outs, kept = block.step(x, context, new, buf, parents=parents)
        ex.check(block)
        assert torch.equal(block.state, state)
        verified_against_prompts(ex, outs, x, trees, before)
        # accept a path of the wanted length, or the longest
        cu = tu.offsets(sizes)
        accepted = []
        for r, (par, want) in enumerate(zip(trees, paths)):
            deepest = max(range(len(par)), key=lambda u: len(tu.path_of(par, u)))
            accepted.append(tu.path_of(par, deepest)[::-1][:want])
        L = max(len(p) for p in accepted)
        path = torch.tensor([p + [-1] * (L - len(p)) for p in accepted], device="cuda")
        block.commit(kept, buf, path, context)
        block.give_back(context, n)
        ex.check(block)
        before = [torch.cat([b, x[cu[r] + torch.tensor(p, dtype=torch.long, device="cuda")]])
                  for r, (b, p) in enumerate(zip(before, accepted))]
        assert context.tolist() == [len(b) for b in before]


def test_a_captured_verification_replays_for_other_trees():
    ex = load_example()
    prompts, nodes = [200, 31], 20
    gen = torch.Generator(device="cuda").manual_seed(4)
    x0 = torch.randn((231, 512), generator=gen, device="cuda").bfloat16()
    block, _ = prompts_of(ex, x0, prompts)
    context, new = tu.i32(prompts), tu.i32([nodes] * 2)
    parents = tu.i32(ex.draft(nodes, 1) + ex.draft(nodes, 2))
    x = torch.randn((2 * nodes, 512), generator=gen, device="cuda").bfloat16()
    buf = block.buffers(2, 2 * nodes)
    block.step(x, context, new, buf, parents=parents)  # takes the pages; libraries settle before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = block.step(x, context, new, buf, parents=parents)
    parents.copy_(tu.i32(tu.parents_of(nodes, "chain") + tu.parents_of(nodes, "flat")))
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    want, _ = block.step(x, context, new, buf, parents=parents)
    ex.check(block)
    assert torch.equal(got, want)
