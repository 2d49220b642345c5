"""GPU: prompt attention, shared prefixes and the 4-bit head together, as examples/sample_prompt.py
runs them: speculative decoding of several samples emits the tokens of plain greedy decoding."""
import importlib.util
import os

import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
I32 = torch.int32


def _example():
    spec = importlib.util.spec_from_file_location("sample_prompt", os.path.join(ROOT, "examples", "sample_prompt.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("length", [200, 256, 31])
def test_samples_are_greedy_continuations_of_their_first_tokens(length):
    ex = _example()
    S, K, V, steps = 3, 3, 2048, 4
    prompt = [(5 + 11 * i * i) % V for i in range(length)]
    rows = ex.decode(ex.Layer(S, V), prompt, K, steps)
    for b in range(S):
        assert 1 + steps <= len(rows[b]) <= 1 + steps * (K + 1)
        # one token a step, over a cache of its own that holds the same prompt, without sharing
        one = ex.Layer(1, V)
        one.prompt(torch.tensor(prompt, device="cuda"))
        for i, t in enumerate(rows[b][:-1]):
            z = one.window(torch.tensor([t], device="cuda"), torch.tensor([length + i], dtype=I32, device="cuda"), 1, share=False)[0].double()
            top = z.topk(2).values
            # Pages of 32 share a scale, which depends on what a window wrote beside the token: logits of
            # the two runs differ by an e4m3 rounding, so a near tie may fall either way.
            if float(top[0] - top[1]) < 0.5:
                break
            assert rows[b][i + 1] == int(z.argmax()), (b, i)


def test_the_prompt_s_attention_is_the_cache_s():
    # the same prompt through the 8-bit cache: keys and values off by 2^-4 of themselves at most (e4m3), which
    # moves a logit by 2^-4 sum |q k| / sqrt(d) and each value by 2^-4: both averaged over many tokens. The bound
    # holds for the mean deviation, which a wrong mask, head or rotation exceeds by far
    ex = _example()
    layer = ex.Layer(1, 2048)
    tokens = torch.arange(300, device="cuda") * 7 % 2048
    a = layer.prompt(tokens)
    n = len(tokens)
    x, qkv = layer.project(tokens)
    h, kv = layer.heads, layer.kv_heads
    cu, zero = torch.tensor([0, n], dtype=I32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    q = sv.spec_kv_append(qkv[:, h:h + kv], qkv[:, h + kv:], layer.kv, zero, cu, layer.table, n, q=qkv[:, :h], cos=layer.cos,
                          sin=layer.sin)
    o, _ = sv.spec_kv_attention(q, layer.kv, zero, cu, layer.table, n)
    b = layer.finish(x, o)
    assert (a - b).abs().mean() <= 2.0 ** -4 * a.abs().mean()


def test_captured_with_its_gradient():
    # forward and gradient recorded by autograd inside a graph, replayed on other values
    g = torch.Generator().manual_seed(1)
    x = torch.randn(150, 8, 64, generator=g).to(torch.bfloat16).cuda()
    cu = torch.tensor([0, 100, 150], dtype=I32, device="cuda")
    leaf, go = x.clone().requires_grad_(), torch.randn(150, 4, 64, generator=g).to(torch.bfloat16).cuda()

    def both(t):
        out, _ = sv.spec_prompt_attention(*t.split([4, 2, 2], 1), cu)
        return out, torch.autograd.grad(out, t, go)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(leaf)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both(leaf)
    with torch.no_grad():
        leaf.copy_(x.flip(0))
    graph.replay()
    ref = both(x.flip(0).contiguous().requires_grad_())
    assert torch.equal(kept[0], ref[0]) and torch.equal(kept[1], ref[1])
