"""Several samples of one prompt, decoded speculatively, with a single attention layer as the target:

    the prompt          q, k, v -> spec_kv_append (keys rotated, into the cache once, for all samples)
                        -> spec_prompt_attention -> spec_lm_head_logits -> a first token for each sample
    a pass              drafts: the layer with its LM head in 4 bits (spec_lm_head_logits_q4);
                        the window: spec_kv_append, spec_kv_attention_shared (the prompt's pages are
                        read once for all samples), spec_lm_head_logits, spec_verify_step

The samples' page tables begin with the prompt's whole pages; a page that the prompt fills in
part is copied for each sample.

    python examples/sample_prompt.py [--samples 4] [--drafts 3] [--steps 6] [--prompt 200] [--vocab 4096]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_30_gb300 as sv  # noqa: E402

I32 = torch.int32


class Layer:
    """A random attention layer, its LM head in bf16 and in 4 bits, and the samples' cache."""

    def __init__(self, samples, vocab, heads=8, kv_heads=2, dim=64, page=32, max_len=1024, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, scale):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)
        self.S, self.heads, self.kv_heads, self.dim, self.page = samples, heads, kv_heads, dim, page
        width = heads * dim
        self.embed = w(vocab, width, scale=1.0)
        self.qkv = w((heads + 2 * kv_heads) * dim, width, scale=width ** -0.5)
        self.out = w(width, width, scale=width ** -0.5)
        self.head = w(vocab, width, scale=2 * width ** -0.5)
        self.head4 = sv.Q4Weight.quantize(self.head, 64)
        pages = -(-max_len // page)
        self.kv = sv.KVCache.empty(samples * pages, page, kv_heads, dim)
        self.table = torch.arange(samples * pages, dtype=I32, device="cuda").view(samples, pages)
        self.cos, self.sin = sv.rope_tables(max_len, dim)
        self.flag = torch.zeros(1, dtype=I32, device="cuda")
        self.groups = torch.tensor([0, samples], dtype=I32, device="cuda")
        self.shared = torch.zeros(1, dtype=I32, device="cuda")

    def project(self, tokens):
        x = self.embed[tokens.long()]
        return x, (x @ self.qkv.T).view(len(x), -1, self.dim)

    def finish(self, x, a, head4=False):
        h = (x + a.reshape(len(x), -1) @ self.out.T).contiguous()
        if head4:
            return sv.spec_lm_head_logits_q4(h, self.head4)
        return sv.spec_lm_head_logits(h, self.head, flag=self.flag)[0]

    def prompt(self, tokens):
        """Logits of a prompt [P]; its keys enter the cache as the first sample's, for all samples."""
        x, qkv = self.project(tokens)
        n, h, kv = len(x), self.heads, self.kv_heads
        cu = torch.tensor([0, n], dtype=I32, device="cuda")
        k, v = qkv[:, h:h + kv], qkv[:, h + kv:]
        rotated = sv.spec_kv_append(k, v, self.kv, torch.zeros(1, dtype=I32, device="cuda"), cu, self.table[:1], n,
                                    q=qkv[:, :h + kv], cos=self.cos, sin=self.sin, flag=self.flag)
        a, _ = sv.spec_prompt_attention(rotated[:, :h], rotated[:, h:], v, cu)
        whole = n // self.page
        self.table[1:, :whole] = self.table[0, :whole]
        if n % self.page:
            for t in self.kv:
                t = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
                t[self.table[1:, whole].long()] = t[self.table[0, whole].long()].clone()
        self.shared.fill_(whole * self.page)
        return self.finish(x, a)

    def window(self, tokens, seq_len, per, head4=False, share=True):
        """Logit rows of `per` new tokens of each sample, packed [S * per]; appends their keys."""
        x, qkv = self.project(tokens)
        h, kv = self.heads, self.kv_heads
        cu = torch.arange(self.S + 1, dtype=I32, device="cuda") * per
        q = sv.spec_kv_append(qkv[:, h:h + kv], qkv[:, h + kv:], self.kv, seq_len, cu, self.table, per, q=qkv[:, :h],
                              cos=self.cos, sin=self.sin, flag=self.flag)
        if share:
            a, _ = sv.spec_kv_attention_shared(q, self.kv, seq_len, cu, self.table, per, self.groups, self.shared)
        else:
            a, _ = sv.spec_kv_attention(q, self.kv, seq_len, cu, self.table, per)
        return self.finish(x, a, head4)


def decode(layer, prompt, drafts, steps, temperature=1.0, seed=0):
    """Samples a first token for each sequence, then greedy speculative decoding; the emitted tokens of each."""
    S, K, dev = layer.S, drafts, "cuda"
    z = layer.prompt(torch.as_tensor(prompt, device=dev))[-1]
    one = torch.ones(S, device=dev)
    none = torch.zeros(S, dtype=I32, device=dev)
    current = sv.spec_sample(z.expand(S, 1, -1).contiguous(), one * temperature, none, one, seed, 0)[:, 0].contiguous()
    seq_len = torch.full((S,), len(prompt), dtype=I32, device=dev)
    offset = torch.zeros(1, dtype=torch.int64, device=dev)
    out, n = torch.empty(S, K + 1, dtype=I32, device=dev), torch.empty(S, dtype=I32, device=dev)
    ws, emitted = sv.Workspace(S, K), [[t] for t in current.tolist()]
    for _ in range(steps):
        tokens = [current]
        for i in range(K):
            tokens.append(layer.window(tokens[-1], seq_len + i, 1, head4=True).argmax(-1).to(I32))
        win = torch.stack(tokens, 1)
        z = layer.window(win.flatten(), seq_len, K + 1).view(S, K + 1, -1)
        sv.spec_verify_step(z, None, win[:, 1:].contiguous(), none.float(), none, one, seed, offset, out, n, ws,
                            next_token=current, seq_len=seq_len)
        for b in range(S):
            emitted[b] += [t for t in out[b].tolist() if t >= 0]
    if int(layer.flag.item()):
        raise RuntimeError("a key could not be stored, or a wait of the LM head ran out")
    return emitted


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--samples", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--steps", type=int, default=6)
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--vocab", type=int, default=4096)
    a = ap.parse_args()
    layer = Layer(a.samples, a.vocab)
    prompt = [(7 + 13 * i * i) % a.vocab for i in range(a.prompt)]
    for b, row in enumerate(decode(layer, prompt, a.drafts, a.steps)):
        print("sample %d: %d tokens in %d steps: %s" % (b, len(row), a.steps, row[:12]))


if __name__ == "__main__":
    main()
