"""GPU: the operators together, as examples/verify_pass.py runs them: greedy speculative
decoding emits the tokens of plain greedy decoding (one token a step through the same
layer), whatever the drafts are, wherever the best token is clear of the second."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("verify_pass", os.path.join(ROOT, "examples", "verify_pass.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("noise", [0.0, 1.0])
def test_speculative_tokens_are_the_greedy_ones(noise):
    ex = _example()
    B, K, V, steps = 3, 3, 2048, 5
    prompts = [[5, 9, 100, 3], [17] * 40, [2, 4]]
    spec = ex.decode(ex.Layer(B, K, V), prompts, steps, noise=noise)
    for b in range(B):
        assert steps <= len(spec[b]) <= steps * (K + 1)
        assert noise or len(spec[b]) > steps           # unperturbed drafts are mostly accepted
        # one token a step, over a cache of its own that holds the same prompt
        one = ex.Layer(1, 1, V)
        seq = torch.zeros(1, dtype=torch.int32, device="cuda")
        z = one.logits(torch.tensor(prompts[b], device="cuda"), seq, torch.tensor([0, len(prompts[b])]))
        t = int(z[-1].argmax())
        for i, (tok, lp) in enumerate(spec[b]):
            seq[0] = len(prompts[b]) + i
            z = one.logits(torch.tensor([t], device="cuda"), seq, torch.tensor([0, 1]))[0].double()
            top = z.topk(2).values
            # Pages of 32 share a scale, which depends on what a window wrote beside the token:
            # logits of the two runs differ by an e4m3 rounding, so a near tie may fall either way.
            if float(top[0] - top[1]) < 0.5:
                break
            assert tok == int(z.argmax()), (b, i)
            assert abs(lp - float(torch.log_softmax(z, 0)[tok])) < 0.5
            t = tok
