"""The example's commit of accepted paths, on the CPU: its calls of the library replaced by what they are defined to do."""
import importlib.util
import os
from types import SimpleNamespace

import pytest
import torch

PAGE = 16


@pytest.fixture()
def example(monkeypatch):
    folder = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")
    spec = importlib.util.spec_from_file_location("tree_step", os.path.join(folder, "tree_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "gdn", SimpleNamespace(gdn_decode_multi=decode_multi, gdn_paged_kv_write=kv_write))
    return mod


def decode_multi(L, q, k, v, g, beta, state, rows, o, dev_status=None):
    """The recurrence over each row's L tokens, token-major rows; states [slot][h][d_v][d_k]."""
    for r, slot in enumerate(rows.tolist()):
        S = state[slot].double()
        for t in range(r * L, (r + 1) * L):
            S = S * g[t].double().exp()[:, None, None]
            fresh = beta[t].double()[:, None] * (v[t].double() - torch.einsum("hvk,hk->hv", S, k[t].double()))
            S = S + torch.einsum("hv,hk->hvk", fresh, k[t].double())
        state[slot] = S.float()


def kv_write(k, v, k_cache, v_cache, slots, dev_status=None):
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            k_cache[s // PAGE, s % PAGE], v_cache[s // PAGE, s % PAGE] = k[i], v[i]


def block_of(example, n, h=2, d=4):
    """A block with what a commit touches, requests of 8 cached tokens on pages 2 r and 2 r + 1."""
    block = object.__new__(example.TreeBlock)
    gen = torch.Generator().manual_seed(n)
    block.page, block.status = PAGE, None
    block.state = torch.randn((n, h, d, d), generator=gen)
    block.k_cache, block.v_cache = (torch.randn((2 * n, PAGE, h, d), generator=gen) for _ in range(2))
    return block


def step_of(sizes, h=2, d=4, seed=0):
    """(kept, buf, context) as a verification of trees of these sizes leaves them."""
    gen = torch.Generator().manual_seed(seed)
    T = sum(sizes)
    kept = tuple(torch.randn((T, h, d), generator=gen) for _ in range(3)) + (
        -torch.rand((T, h), generator=gen), torch.rand((T, h), generator=gen))
    cu = [sum(sizes[:r]) for r in range(len(sizes) + 1)]
    slots = [2 * r * PAGE + 8 + u for r, m in enumerate(sizes) for u in range(m)]
    buf = {"cu": torch.tensor(cu, dtype=torch.int32), "slots": torch.tensor(slots, dtype=torch.int32),
           "rows": torch.arange(len(sizes), dtype=torch.int32)}
    return kept, buf, torch.full((len(sizes),), 8, dtype=torch.int32)


def committed(block, kept, buf, paths):
    """States and caches with each path's nodes one behind the other."""
    state, caches = block.state.clone(), [block.k_cache.clone(), block.v_cache.clone()]
    for r, path in enumerate(paths):
        first = int(buf["cu"][r])
        tok = [first + u for u in path]
        decode_multi(len(path), *(x[tok] for x in kept), state, torch.tensor([r]), None)
        for i, t in enumerate(tok):
            to, at = int(buf["slots"][first + i]), int(buf["slots"][t])
            for new, old in zip(caches, (block.k_cache, block.v_cache)):
                new[to // PAGE, to % PAGE] = old[at // PAGE, at % PAGE]
    return state, *caches


def commit(example, sizes, paths, spoil=()):
    block = block_of(example, len(sizes))
    kept, buf, context = step_of(sizes)
    for t in spoil:
        for x in kept:
            x[t] = float("nan")
    want = committed(block, kept, buf, paths)
    L = max([len(p) for p in paths], default=0)
    path = torch.tensor([p + [-1] * (L - len(p)) for p in paths], dtype=torch.int64).reshape(len(paths), L)
    block.commit(kept, buf, path, context)
    assert context.tolist() == [8 + len(p) for p in paths]
    torch.testing.assert_close(block.state, want[0], rtol=0, atol=0)
    assert torch.equal(block.k_cache, want[1]) and torch.equal(block.v_cache, want[2])


@pytest.mark.parametrize("sizes,paths", [
    ([5, 7], [[0, 2, 4], [1, 6]]), ([4, 2, 0], [[0, 1, 3], [0], []]), ([0, 3], [[], [0, 2]]), ([3, 0, 0, 2], [[2], [], [], []]),
    ([0, 0], [[], []]), ([3, 1], [[], []]), ([1], [[0]])])
def test_paths_of_any_length(example, sizes, paths):
    commit(example, sizes, paths)


@pytest.mark.parametrize("sizes,paths,spoil", [
    ([5, 7], [[1, 2], [0, 3, 5]], [0]), ([5, 7], [[], [0, 3, 5]], [0, 3]), ([0, 4, 3], [[], [1], [2, 1]], [0, 2, 4])])
def test_rejected_nodes_that_are_not_finite(example, sizes, paths, spoil):
    # a token that fills up a shorter path is no accepted one, whatever that holds
    commit(example, sizes, paths, spoil)
