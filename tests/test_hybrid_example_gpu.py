"""The example's serving steps: decode tokens through the captured step against the same tokens as part of the prompt."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def load_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_step.py")
    spec = importlib.util.spec_from_file_location("hybrid_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_decoded_tokens_match_the_same_tokens_as_prompts():
    ex = load_example()
    prompts, steps = [116, 321, 64], 5
    _, outs, (x, fed, _) = ex.serve(ex.HybridBlock(), prompts, steps)
    # all at once: each request's prompt followed by its later tokens
    parts, at = [], 0
    for r, p in enumerate(prompts):
        parts += [x[at:at + p], fed[:, r]]
        at += p
    whole = torch.cat(parts)
    lens = [p + steps for p in prompts]
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    block = ex.HybridBlock()
    new = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref = block.step(whole, torch.zeros_like(new), new, block.buffers(len(lens), whole.shape[0]), cu).float()
    assert block.status.item() == 0
    for s in range(steps):
        for r in range(len(prompts)):
            got, want = outs[s][r].float(), ref[cu[r + 1] - steps + s]
            # the recurrence in one form against the other and bf16 in between: 2e-2 of the values' size each, as the
            # two layers are held to by themselves
            assert (got - want).abs().max() <= 4e-2 * (1 + want.abs().max()), (s, r)
