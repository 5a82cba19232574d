"""The example's commit of requests without a draft, or without an accepted node."""
import pytest
import torch

from tests import tree_util as tu
from tests.test_tree_example_gpu import load_example, prompts_of, verified_against_prompts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,lengths", [([9, 5, 0], [2, 1, 0]), ([0, 12, 3], [0, 3, 0])])
def test_requests_without_nodes(sizes, lengths):
    ex = load_example()
    prompts = [70, 33, 19]
    gen = torch.Generator(device="cuda").manual_seed(5)
    x0 = torch.randn((sum(prompts), 512), generator=gen, device="cuda").bfloat16()
    block, _ = prompts_of(ex, x0, prompts)
    context, before = tu.i32(prompts), list(x0.split(prompts))
    trees = [ex.draft(m, r) for r, m in enumerate(sizes)]
    x = torch.randn((sum(sizes), 512), generator=gen, device="cuda").bfloat16()
    buf, state = block.buffers(3, sum(sizes)), block.state.clone()
    _, kept = block.step(x, context, tu.i32(sizes), buf, parents=tu.i32(sum(trees, [])))
    paths = []
    for par, most in zip(trees, lengths):
        deepest = max(range(len(par)), key=lambda u: len(tu.path_of(par, u)), default=-1)
        paths.append(tu.path_of(par, deepest)[::-1][:most])
    L = max(len(p) for p in paths)
    block.commit(kept, buf, torch.tensor([p + [-1] * (L - len(p)) for p in paths], device="cuda"), context)
    block.give_back(context, 3)
    ex.check(block)
    assert context.tolist() == [a + len(p) for a, p in zip(prompts, paths)]
    for r, p in enumerate(paths):
        assert torch.equal(block.state[r], state[r]) == (not p)
    # the next trees see what was accepted
    cu = tu.offsets(sizes)
    before = [torch.cat([b, x[cu[r] + torch.tensor(p, dtype=torch.long, device="cuda")]])
              for r, (b, p) in enumerate(zip(before, paths))]
    trees, new = [ex.draft(7, 9 + r) for r in range(3)], tu.i32([7] * 3)
    x = torch.randn((21, 512), generator=gen, device="cuda").bfloat16()
    outs, _ = block.step(x, context, new, block.buffers(3, 21), parents=tu.i32(sum(trees, [])))
    ex.check(block)
    verified_against_prompts(ex, outs, x, trees, before)


def test_a_rejected_node_that_is_not_finite():
    ex = load_example()
    prompts, sizes = [70, 33], [5, 7]
    gen = torch.Generator(device="cuda").manual_seed(6)
    x0 = torch.randn((sum(prompts), 512), generator=gen, device="cuda").bfloat16()
    x = torch.randn((sum(sizes), 512), generator=gen, device="cuda").bfloat16()
    trees, states = [[-1, -1, 1, 0, 2], [-1] * 7], []
    for spoil in (False, True):
        block, _ = prompts_of(ex, x0, prompts)
        context, buf = tu.i32(prompts), block.buffers(2, sum(sizes))
        fed = x.clone()
        if spoil:
            fed[0], fed[6:] = float("nan"), float("inf")
        _, kept = block.step(fed, context, tu.i32(sizes), buf, parents=tu.i32(sum(trees, [])))
        block.commit(kept, buf, torch.tensor([[1, 2, 4], [0, -1, -1]], device="cuda"), context)
        ex.check(block)
        states.append(block.state[:2].clone())
    assert torch.isfinite(states[1]).all() and torch.equal(*states)
