"""One verify pass of speculative decoding with a single attention layer as the target:

    hidden states of the window (the last emitted token and K drafted ones)
      -> q, k, v             one projection
      -> spec_kv_append      keys and values into the paged 8-bit cache, rotated
      -> spec_kv_attention   the window's queries over the cache
      -> spec_lm_head_logits, spec_verify_step
      -> spec_token_logprobs of the emitted tokens, with alternatives

The step keeps its lengths on the device: spec_verify_step advances seq_len by the
tokens it emitted, and the next window overwrites the places of rejected drafts.

    python examples/verify_pass.py [--batch 4] [--drafts 3] [--steps 6] [--vocab 4096]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_30_gb300 as sv  # noqa: E402


class Layer:
    """A random attention layer and its cache; drafts come from the layer's own logits, perturbed."""

    def __init__(self, batch, drafts, vocab, heads=8, kv_heads=2, dim=64, page=32, max_len=512, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, scale):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)
        self.B, self.K, self.heads, self.kv_heads, self.dim = batch, drafts, heads, kv_heads, dim
        width = heads * dim
        self.embed = w(vocab, width, scale=1.0)
        self.qkv = w((heads + 2 * kv_heads) * dim, width, scale=width ** -0.5)
        self.out = w(width, width, scale=width ** -0.5)
        self.head = w(vocab, width, scale=2 * width ** -0.5)
        pages = -(-max_len // page)
        self.kv = sv.KVCache.empty(batch * pages, page, kv_heads, dim)
        self.table = torch.arange(batch * pages, dtype=torch.int32, device="cuda").view(batch, pages)
        self.cos, self.sin = sv.rope_tables(max_len, dim)
        self.flag = torch.zeros(1, dtype=torch.int32, device="cuda")

    def logits(self, tokens, seq_len, cu):
        """Logit rows of packed tokens [N] at positions seq_len[b], seq_len[b] + 1, ...; appends their keys."""
        x = self.embed[tokens.long()]
        n, most = x.shape[0], int(max(cu[1:] - cu[:-1]))
        cu = torch.as_tensor(cu, dtype=torch.int32).cuda()
        qkv = (x @ self.qkv.T).view(n, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = sv.spec_kv_append(k, v, self.kv, seq_len, cu, self.table, most, q=q, cos=self.cos, sin=self.sin, flag=self.flag)
        a, _ = sv.spec_kv_attention(q, self.kv, seq_len, cu, self.table, most)
        h = x + a.reshape(n, -1) @ self.out.T
        return sv.spec_lm_head_logits(h.contiguous(), self.head, flag=self.flag)[0]


def decode(layer, prompts, steps, seed=0, noise=0.5):
    """Greedy speculative decoding; returns, for each sequence, its emitted (token, log-probability) pairs."""
    B, K = layer.B, layer.K
    dev, i32 = "cuda", torch.int32
    seq_len = torch.zeros(B, dtype=i32, device=dev)
    cu = torch.tensor([0] + [len(p) for p in prompts]).cumsum(0)
    z = layer.logits(torch.tensor(sum(prompts, []), device=dev), seq_len, cu)
    current = z[(cu[1:] - 1).to(dev)].argmax(-1).to(i32)          # the first token after each prompt
    seq_len += torch.tensor([len(p) for p in prompts], dtype=i32, device=dev)
    g = torch.Generator(device=dev).manual_seed(seed)
    zero, one = torch.zeros(B, device=dev), torch.ones(B, device=dev)
    none, offset = torch.zeros(B, dtype=i32, device=dev), torch.zeros(1, dtype=torch.int64, device=dev)
    out, n = torch.empty(B, K + 1, dtype=i32, device=dev), torch.empty(B, dtype=i32, device=dev)
    ws, emitted = sv.Workspace(B, K), [[] for _ in range(B)]
    window = torch.arange(B + 1) * (K + 1)
    for _ in range(steps):
        # drafts: greedy tokens of perturbed logits, one after the other (the cache is overwritten below)
        tokens = [current]
        for i in range(K):
            z = layer.logits(tokens[-1], seq_len + i, torch.arange(B + 1))
            z = z + noise * torch.randn(z.shape, generator=g, device=dev)
            tokens.append(z.argmax(-1).to(i32))
        win = torch.stack(tokens, 1)
        z = layer.logits(win.flatten(), seq_len, window).view(B, K + 1, -1)
        sv.spec_verify_step(z, None, win[:, 1:].contiguous(), zero, none, one, seed, offset, out, n, ws,
                            next_token=current, seq_len=seq_len)
        scored = sv.spec_token_logprobs(z, out, top_n=3)
        for b in range(B):
            emitted[b] += [(t, lp) for t, lp in zip(out[b].tolist(), scored.logprob[b].tolist()) if t >= 0]
    if int(layer.flag.item()):
        raise RuntimeError("a key could not be stored, or a wait of the LM head ran out")
    return emitted


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--steps", type=int, default=6)
    ap.add_argument("--vocab", type=int, default=4096)
    a = ap.parse_args()
    layer = Layer(a.batch, a.drafts, a.vocab)
    prompts = [[(7 * b + 3 * i) % a.vocab for i in range(5 + 9 * b)] for b in range(a.batch)]
    for b, row in enumerate(decode(layer, prompts, a.steps)):
        print("sequence %d: %d tokens in %d steps, mean log-probability %.3f: %s" % (
            b, len(row), a.steps, sum(lp for _, lp in row) / len(row), [t for t, _ in row][:12]))


if __name__ == "__main__":
    main()
