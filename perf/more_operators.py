"""The cases on which the operators of prompts, shared prefixes and 4-bit LM heads are timed.

Three operators, each with the plain torch form it is compared with:

* prompt attention: causal attention over packed prompts of different lengths, with
  grouped heads and sliding windows, and its gradient with respect to queries, keys and
  values;
* attention on a shared prefix: windows of new tokens over a paged cache held in 8 bits
  (e4m3 codes, a scale for each page and head), in which the sequences of a group have
  their leading pages in common;
* the LM head in 4 bits: logits of a few hidden states over a vocabulary whose weights
  are codes of 0..15 with a scale and a bias for each group along the hidden dimension.

`own` selects the framework's calls; otherwise the plain forms run.
"""
import math
import random

import torch

own = False

VOCAB = 151_936          # the vocabulary of the repository's workloads
E4M3_MAX = 448.0


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # a few short prompts arriving together: latency counts
        dict(name="prompt 3 short", op="prompt", batch=3, tokens=70, ragged=True, heads=16, kv_heads=2, dim=128, window=0),
        # prompts of many lengths in one call
        dict(name="prompt 24 packed", op="prompt", batch=24, tokens=1500, ragged=True, heads=32, kv_heads=8, dim=128, window=0),
        # two long documents
        dict(name="prompt 2 long", op="prompt", batch=2, tokens=8192, ragged=False, heads=32, kv_heads=8, dim=128, window=0),
        # narrow heads without sharing, a layer with a sliding window
        dict(name="prompt 8 in a window", op="prompt", batch=8, tokens=4001, ragged=True, heads=12, kv_heads=12, dim=64, window=1000),
        # training a draft head on short ragged texts: odd lengths, seven query heads to a kv head
        dict(name="gradient 5 short", op="gradient", batch=5, tokens=333, ragged=True, heads=14, kv_heads=2, dim=64, window=0),
        # a training batch of packed documents
        dict(name="gradient 12 packed", op="gradient", batch=12, tokens=2500, ragged=True, heads=32, kv_heads=8, dim=128, window=0),
        # four samples of one prompt: latency counts
        dict(name="shared 4 samples", op="shared", groups=1, batch=4, tokens=2, ragged=False, heads=16, kv_heads=8, dim=128,
             page=64, prefix=3000, context=200),
        # the serving batch behind one long system prompt: 64 sequences, 5 tokens each
        dict(name="shared 64 windows", op="shared", groups=1, batch=64, tokens=5, ragged=False, heads=32, kv_heads=8, dim=128,
             page=64, prefix=8000, context=600),
        # six prompts sampled 16 times each, single tokens, narrow heads, small pages
        dict(name="shared 6 prompts", op="shared", groups=6, batch=96, tokens=1, ragged=False, heads=24, kv_heads=4, dim=64,
             page=16, prefix=5000, context=1500),
        # one drafted token: a single row
        dict(name="head 1 row", op="head", rows=1, vocab=VOCAB, dim=1024, group=64),
        # a verify window of one sequence through a wide head
        dict(name="head 5 rows", op="head", rows=5, vocab=VOCAB, dim=4096, group=128),
        # a batch of drafted tokens, an odd vocabulary, small groups
        dict(name="head 40 rows", op="head", rows=40, vocab=50_257, dim=2048, group=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "gradient", "gradient", "shared", "shared", "head"])
    if op == "head":
        dim = 64 * rng.randint(4, 64)
        return dict(op=op, rows=_log(rng, 1, 64), vocab=_log(rng, 2000, min(260_000, 6e8 / dim)), dim=dim,
                    group=rng.choice([g for g in (32, 64, 128) if dim % g == 0]))
    kv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, heads=kv * rng.choice([1, 2, 3, 4, 7, 8]), kv_heads=kv, dim=rng.choice([64, 128]))
    if op in ("prompt", "gradient"):
        c |= dict(tokens=_log(rng, 1, 8000 if op == "prompt" else 4000), ragged=rng.random() < 0.7)
        pairs = (4e9 if op == "prompt" else 2e9) / c["heads"] / c["tokens"] ** 2
        c["batch"] = _log(rng, 1, max(1.5, min(200, pairs, 40_000 / c["tokens"])))
        c["window"] = rng.choice([0, 0, 0, 100, 1000])
        return c
    c |= dict(page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.4, tokens=_log(rng, 1, 12), prefix=_log(rng, 30, 20_000),
              context=_log(rng, 1, 3000))
    token = c["tokens"] * c["heads"] * c["dim"] * (c["prefix"] + c["context"])
    c["batch"] = _log(rng, 2, max(3, min(128, 1e10 / token, 1e6 / (c["prefix"] + c["context"]))))
    c["groups"] = min(c["batch"], rng.choice([1, 1, 2, 5]))
    return c


def _prompts(case):
    """Tokens of each prompt: fixed by the case alone."""
    r = random.Random("%(batch)d %(tokens)d %(heads)d" % case)
    n, t = case["batch"], case["tokens"]
    new = [r.randint(1, t) for _ in range(n)] if case["ragged"] else [t] * n
    new[0] = t
    return new


def _sequences(case):
    """Group of each sequence, prefix of each group, own cached tokens and new tokens of each sequence."""
    r = random.Random("%(batch)d %(tokens)d %(prefix)d %(context)d" % case)
    n, g = case["batch"], case["groups"]
    of = sorted(list(range(g)) + [r.randrange(g) for _ in range(n - g)])
    prefix = [r.randint(case["prefix"] // 2, case["prefix"]) for _ in range(g)]
    prefix[0] = case["prefix"]
    prefix = [-(-p // case["page"]) * case["page"] for p in prefix]      # whole pages are shared
    ctx = [r.randint(0, case["context"]) for _ in range(n)]
    new = [r.randint(0, case["tokens"]) for _ in range(n)] if case["ragged"] else [case["tokens"]] * n
    new[0] = case["tokens"]
    return of, prefix, ctx, new


def _pairs(t, window):
    """(query, key) pairs of a causal prompt of t tokens."""
    w = min(window, t) if window else t
    return w * (w + 1) // 2 + (t - w) * w


def work(case):
    if case["op"] == "head":
        m, v, d = case["rows"], case["vocab"], case["dim"]
        return {"bytes": v * d // 2 + 4 * v * (d // case["group"]) + 2 * m * d + 4 * m * v, "flops": 2 * m * v * d}
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("prompt", "gradient"):
        new = _prompts(case)
        n, pairs = sum(new), sum(_pairs(t, case["window"]) for t in new)
        if case["op"] == "prompt":
            return {"bytes": 4 * n * (h + kv) * d + 4 * n * h, "flops": 4 * pairs * h * d}
        # q, k, v, out, grad_out and lse are read, three gradients written
        return {"bytes": 2 * n * d * (3 * h + 2 * kv) + 4 * n * h + 2 * n * d * (h + 2 * kv), "flops": 10 * pairs * h * d}
    of, prefix, ctx, new = _sequences(case)
    keys = sum(prefix) + sum(c + t for c, t in zip(ctx, new) if t)
    pages = sum(p // case["page"] for p in prefix) + sum(-(-(c + t) // case["page"]) for c, t in zip(ctx, new) if t)
    pairs = sum(t * (prefix[g] + c) + t * (t + 1) // 2 for g, c, t in zip(of, ctx, new))
    n = sum(new)
    return {"bytes": keys * kv * 2 * d + pages * kv * 8 + n * h * (4 * d + 4), "flops": 4 * pairs * h * d}


# --- inputs ------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cu(new):
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    return cu


def _codes(x):
    """Values [..., page, dim] in e4m3 with a power-of-two scale for each page and head."""
    top = x.abs().amax((-2, -1))
    s = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))
    return (x / s[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def _prepare_head(case, g):
    v, d, group = case["vocab"], case["dim"], case["group"]
    w = torch.randn(v, d // group, group, generator=g, device="cuda")
    w *= torch.exp(0.3 * torch.randn(v, 1, 1, generator=g, device="cuda")) * d ** -0.5    # tokens have different norms
    lo, hi = w.amin(2, keepdim=True), w.amax(2, keepdim=True)
    scale, bias = ((hi - lo) / 15).to(torch.bfloat16), lo.to(torch.bfloat16)
    q = ((w - bias.float()) / scale.float()).round().clamp(0, 15).to(torch.uint8).view(v, d)
    del w
    codes = q[:, 0::2] | q[:, 1::2] << 4           # the first of two neighbours in the low half of a byte
    hidden = torch.randn(case["rows"], d, generator=g, device="cuda").to(torch.bfloat16)
    return dict(case=case, hidden=hidden, codes=codes, scale=scale.view(v, -1), bias=bias.view(v, -1))


def _prepare_prompt(case, g):
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    new = _prompts(case)
    n, cu = sum(new), _cu(new)
    qkv = torch.randn(n, h + 2 * kv, d, generator=g, device="cuda")
    qkv[:, :h + kv] *= torch.exp(0.3 * torch.randn(1, h + kv, d, generator=g, device="cuda"))   # strong channels
    qkv = qkv.to(torch.bfloat16)                                                                # one projection's output
    q, k, v = qkv.split([h, kv, kv], 1)
    s = dict(case=case, q=q, k=k, v=v, cu=torch.tensor(cu, device="cuda", dtype=torch.int32), most=max(new))
    if case["op"] == "gradient":
        s["grad_out"] = torch.randn(n, h, d, generator=g, device="cuda").to(torch.bfloat16)
        out, lse = [], []
        for a, b in zip(cu[:-1], cu[1:]):              # what the forward pass left
            o, m = _one_prompt(q[a:b].float(), k[a:b].float(), v[a:b].float(), case)
            out.append(o.to(torch.bfloat16))
            lse.append(m)
        s["out"], s["lse"] = torch.cat(out), torch.cat(lse)
    return s


def _seen(t, window):
    i = torch.arange(t, device="cuda")
    see = i[:, None] >= i
    return see & (i[:, None] - i < window) if window else see


def _one_prompt(q, k, v, case):
    """out [t, h, d] and lse [t, h] of one prompt."""
    t, h, d = q.shape
    kv = k.shape[1]
    q = q.view(t, kv, h // kv, d).permute(1, 2, 0, 3).reshape(kv, -1, d)
    a = torch.matmul(q, k.permute(1, 2, 0)) * d ** -0.5
    a = a.view(kv, h // kv, t, t).masked_fill_(~_seen(t, case["window"]), -math.inf)
    m = torch.logsumexp(a, 3, keepdim=True)
    o = torch.matmul(a.sub_(m).exp_().view(kv, -1, t), v.transpose(0, 1)).view(h, t, d)
    return o.transpose(0, 1), m.view(h, t).T


def _prepare_shared(case, g):
    of, prefix, ctx, new = _sequences(case)
    b, kv, d, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    own_pages = [-(-(c + t) // page) for c, t in zip(ctx, new)]
    pool = sum(prefix) // page + sum(own_pages) + 3
    order = torch.randperm(pool, generator=g, device="cuda").tolist()
    at, lead = 0, []
    for p in prefix:
        lead.append(order[at:at + p // page])
        at += p // page
    per = max(prefix[i] // page + n for i, n in zip(of, own_pages))
    table = []
    for i, n in zip(of, own_pages):
        row = lead[i] + order[at:at + n]
        at += n
        table.append(row + [-1] * (per - len(row)))
    dev = dict(device="cuda", dtype=torch.int32)
    total = [prefix[i] + c for i, c in zip(of, ctx)]
    s = dict(case=case, seq_len=torch.tensor(total, **dev), cu=torch.tensor(_cu(new), **dev), table=torch.tensor(table, **dev),
             max_tokens=max(new), shared_len=torch.tensor(prefix, **dev),
             longest=max(sum(t for j, t in zip(of, new) if j == i) for i in range(case["groups"])),
             cu_groups=torch.tensor(_cu([of.count(i) for i in range(case["groups"])]), **dev))
    gain = torch.exp(0.5 * torch.randn(kv, 1, d, generator=g, device="cuda"))     # keys have strong channels
    s["k_cache"], s["k_scale"] = _codes(gain * torch.randn(pool, kv, page, d, generator=g, device="cuda"))
    v = torch.randn(pool, kv, page, d, generator=g, device="cuda")
    s["v_cache"], s["v_scale"] = _codes(v * torch.exp(0.7 * torch.randn(pool, kv, 1, 1, generator=g, device="cuda")))
    del v
    for i, (c, t) in enumerate(zip(total, new)):       # what lies past the end is never looked at: NaN codes
        if (c + t) % page and own_pages[i]:
            for x in (s["k_cache"], s["v_cache"]):
                x.view(torch.uint8)[table[i][(c + t) // page], :, (c + t) % page:] = 0x7F
    q = torch.randn(sum(new), case["heads"], d, generator=g, device="cuda")
    s["q"] = (q * torch.exp(0.3 * torch.randn(sum(new), case["heads"], 1, generator=g, device="cuda"))).to(torch.bfloat16)
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "head":
        return _prepare_head(case, g)
    return _prepare_shared(case, g) if case["op"] == "shared" else _prepare_prompt(case, g)


# --- the plain forms ---------------------------------------------------------

def _plain_head(s):
    v, d = s["codes"].shape[0], s["hidden"].shape[1]
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(v, -1, s["case"]["group"]).float()
    w = (q * s["scale"].float()[..., None] + s["bias"].float()[..., None]).view(v, d)
    return torch.matmul(s["hidden"].float(), w.T)


class _Padded:
    """Rows of packed prompts as [batch, heads, most, ...] and back."""

    def __init__(self, s):
        n, b = s["q"].shape[0], s["case"]["batch"]
        cu = s["cu"].long()
        self.b, self.t = b, s["most"]
        self.of = torch.repeat_interleave(torch.arange(b, device="cuda"), cu[1:] - cu[:-1], output_size=n)
        self.i = torch.arange(n, device="cuda") - cu[self.of]

    def pad(self, x):
        y = torch.zeros(self.b, self.t, *x.shape[1:], device="cuda")
        y[self.of, self.i] = x.float()
        return y.transpose(1, 2)

    def pack(self, y):
        return y.transpose(1, 2)[self.of, self.i]


def _plain_prompt(s):
    c, p = s["case"], _Padded(s)
    b, h, kv, d, t = c["batch"], c["heads"], c["kv_heads"], c["dim"], s["most"]
    q, k, v = p.pad(s["q"]), p.pad(s["k"]), p.pad(s["v"])
    a = torch.matmul(q.reshape(b, kv, -1, d), k.transpose(2, 3)).mul_(d ** -0.5).view(b, h, t, t)
    a.masked_fill_(~_seen(t, c["window"]), -math.inf)
    m = a.amax(3, keepdim=True)
    a = a.sub_(m).exp_()
    total = a.sum(3, keepdim=True)
    o = torch.matmul(a.view(b, kv, -1, t), v).view(b, h, t, d) / total
    return dict(out=p.pack(o).to(torch.bfloat16), lse=p.pack((m + total.log())[..., 0]))


def _plain_gradient(s):
    c, p = s["case"], _Padded(s)
    b, h, kv, d, t = c["batch"], c["heads"], c["kv_heads"], c["dim"], s["most"]
    q, k, v, go = p.pad(s["q"]), p.pad(s["k"]), p.pad(s["v"]), p.pad(s["grad_out"])
    lse, delta = p.pad(s["lse"]), (go * p.pad(s["out"])).sum(3)
    q, go = q.reshape(b, kv, -1, d), go.reshape(b, kv, -1, d)
    w = torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5).view(b, h, t, t)
    w = w.sub_(lse[..., None]).masked_fill_(~_seen(t, c["window"]), -math.inf).exp_().view(b, kv, -1, t)
    gv = torch.matmul(w.transpose(2, 3), go)
    ds = torch.matmul(go, v.transpose(2, 3)).sub_(delta.reshape(b, kv, -1, 1)).mul_(w).mul_(d ** -0.5)
    gq = torch.matmul(ds, k).view(b, h, t, d)
    gk = torch.matmul(ds.transpose(2, 3), q)
    ty = torch.bfloat16
    return dict(grad_q=p.pack(gq).to(ty), grad_k=p.pack(gk).to(ty), grad_v=p.pack(gv).to(ty))


def _plain_shared(s):
    """The prefix of each group once, for all of the group's rows; then each sequence's own tokens; then their join."""
    c = s["case"]
    b, h, kv, d, page, groups = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"], c["groups"]
    n, t, longest, r = s["q"].shape[0], s["max_tokens"], s["longest"], c["heads"] // c["kv_heads"]
    cu, cg, shared, ctx = s["cu"].long(), s["cu_groups"].long(), s["shared_len"].long(), s["seq_len"].long()
    rows = torch.arange(n, device="cuda")
    of = torch.repeat_interleave(torch.arange(b, device="cuda"), cu[1:] - cu[:-1], output_size=n)
    group = torch.repeat_interleave(torch.arange(groups, device="cuda"), cg[1:] - cg[:-1], output_size=b)
    table = s["table"].long().clamp(min=0)
    wide = table.shape[1] * page

    def values(codes, scale, pages, live):
        x = codes[pages].float() * scale[pages][..., None, None]          # [batch, pages, kv, page, d]
        x = x.transpose(1, 2).reshape(pages.shape[0], kv, -1, d)
        return torch.where(live[:, None, :, None], x, 0.0)

    def part(q, see, pages, live):
        """Frame, sum and weighted values of queries [batch, kv, rows, d]."""
        a = torch.matmul(q, values(s["k_cache"], s["k_scale"], pages, live).transpose(2, 3)) * d ** -0.5
        a = a.masked_fill(~see, -math.inf)
        m = a.amax(3, keepdim=True).clamp(min=-1e30)
        a = torch.exp(a - m)
        return m, a.sum(3, keepdim=True), torch.matmul(a, values(s["v_cache"], s["v_scale"], pages, live))

    # prefixes: rows of a group one after the other
    first = cu[cg[:-1]]
    at = rows - first[group[of]]
    q = torch.zeros(groups, longest, h, d, device="cuda")
    q[group[of], at] = s["q"].float()
    q = q.view(groups, longest, kv, r, d).permute(0, 2, 1, 3, 4).reshape(groups, kv, longest * r, d)
    live = torch.arange(wide, device="cuda") < shared[:, None]
    m1, l1, o1 = part(q, live[:, None, None], table[cg[:-1]], live)

    def back1(x):
        return x.view(groups, kv, longest, r, -1).permute(0, 2, 1, 3, 4).reshape(groups, longest, h, -1)[group[of], at]

    # own tokens: a sequence's row of the table from the prefix on
    i = rows - cu[of]
    q = torch.zeros(b, t, h, d, device="cuda")
    q[of, i] = s["q"].float()
    q = q.view(b, t, kv, r, d).permute(0, 2, 1, 3, 4).reshape(b, kv, t * r, d)
    span = -(-(c["context"] + c["tokens"]) // page)
    lead = shared[group] // page
    j = lead[:, None] + torch.arange(span, device="cuda")
    pages = table.gather(1, j.clamp(max=table.shape[1] - 1))
    pos = shared[group][:, None] + torch.arange(span * page, device="cuda")
    see = pos[:, None, :] <= ctx[:, None, None] + torch.arange(t, device="cuda")[:, None]
    see = see[:, None, :, None].expand(b, 1, t, r, span * page).reshape(b, 1, t * r, span * page)
    live = pos < (ctx + cu[1:] - cu[:-1])[:, None]
    m2, l2, o2 = part(q, see, pages, live)

    def back2(x):
        return x.view(b, kv, t, r, -1).permute(0, 2, 1, 3, 4).reshape(b, t, h, -1)[of, i]

    m1, l1, o1, m2, l2, o2 = back1(m1), back1(l1), back1(o1), back2(m2), back2(l2), back2(o2)
    m = torch.maximum(m1, m2)
    f1, f2 = torch.exp(m1 - m), torch.exp(m2 - m)
    total = l1 * f1 + l2 * f2
    return dict(out=((o1 * f1 + o2 * f2) / total).to(torch.bfloat16), lse=(m + total.log())[..., 0])


def run(s):
    c = s["case"]
    if own:
        import speculative_decoding_verification_30_gb300 as sv
    if c["op"] == "head":
        if own:
            return sv.spec_lm_head_logits_q4(s["hidden"], sv.Q4Weight(s["codes"], s["scale"], s["bias"]))
        return _plain_head(s)
    if c["op"] == "prompt":
        if own:
            out, lse = sv.spec_prompt_attention(s["q"], s["k"], s["v"], s["cu"], window=c["window"])
            return dict(out=out, lse=lse)
        return _plain_prompt(s)
    if c["op"] == "gradient":
        if own:
            gq, gk, gv = sv.spec_prompt_attention_backward(s["grad_out"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["cu"],
                                                           window=c["window"])
            return dict(grad_q=gq, grad_k=gk, grad_v=gv)
        return _plain_gradient(s)
    if own:
        kv = sv.KVCache(s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"])
        out, lse = sv.spec_kv_attention_shared(s["q"], kv, s["seq_len"], s["cu"], s["table"], s["max_tokens"], s["cu_groups"],
                                               s["shared_len"])
        return dict(out=out, lse=lse)
    return _plain_shared(s)


# --- the definitions in 64 bits ----------------------------------------------

def _exact_head(s):
    c, rows = s["case"], []
    h = s["hidden"].double()
    for a in range(0, c["vocab"], 16_384):
        codes = s["codes"][a:a + 16_384]
        w = torch.empty(codes.shape[0], c["dim"], device="cuda", dtype=torch.float64)
        w[:, 0::2] = (codes % 16).double()
        w[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
        each = torch.arange(c["dim"], device="cuda") // c["group"]
        w = w * s["scale"][a:a + 16_384].double()[:, each] + s["bias"][a:a + 16_384].double()[:, each]
        rows.append(h @ w.T)
    return torch.cat(rows, 1)


def _exact_prompts(s):
    c, gradient = s["case"], s["case"]["op"] == "gradient"
    h, kv, d = c["heads"], c["kv_heads"], c["dim"]
    if sum(t * t for t in _prompts(c)) * h * d * (10 if gradient else 4) > 8e12:
        return None
    ty = dict(device="cuda", dtype=torch.float64)
    n = s["q"].shape[0]
    cu = s["cu"].tolist()
    res = [torch.zeros(n, h, d, **ty), torch.zeros(n, h, **ty)] if not gradient else \
        [torch.zeros(n, h, d, **ty), torch.zeros(n, kv, d, **ty), torch.zeros(n, kv, d, **ty)]
    for a, e in zip(cu[:-1], cu[1:]):
        i = torch.arange(e - a, device="cuda")
        hidden = i[None, :] > i[:, None]
        if c["window"]:
            hidden |= i[None, :] <= i[:, None] - c["window"]
        for x in range(h):
            y = x // (h // kv)
            q, k, v = s["q"][a:e, x].double(), s["k"][a:e, y].double(), s["v"][a:e, y].double()
            z = (q @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            p = torch.softmax(z, 1)
            if not gradient:
                res[0][a:e, x] = p @ v
                res[1][a:e, x] = torch.logsumexp(z, 1)
                continue
            go = s["grad_out"][a:e, x].double()
            dp = go @ v.T
            dz = p * (dp - (dp * p).sum(1, keepdim=True)) / math.sqrt(d)
            res[0][a:e, x] = dz @ k
            res[1][a:e, y] += dz.T @ q
            res[2][a:e, y] += p.T @ go
    return dict(zip(("grad_q", "grad_k", "grad_v") if gradient else ("out", "lse"), res))


def _exact_shared(s):
    """Every sequence by itself, over all of its row of the page table."""
    c = s["case"]
    h, kv, d, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    ctx, cu = s["seq_len"].tolist(), s["cu"].tolist()
    outs, norms = [], []
    for b in range(c["batch"]):
        t = cu[b + 1] - cu[b]
        if not t:
            continue
        end = ctx[b] + t
        pages = s["table"][b, :-(-end // page)].long()
        o = torch.empty(t, h, d, device="cuda", dtype=torch.float64)
        norm = torch.empty(t, h, device="cuda", dtype=torch.float64)
        for j in range(kv):
            key = (s["k_cache"][pages, j].double() * s["k_scale"][pages, j].double()[:, None, None]).reshape(-1, d)[:end]
            val = (s["v_cache"][pages, j].double() * s["v_scale"][pages, j].double()[:, None, None]).reshape(-1, d)[:end]
            heads = slice(j * (h // kv), (j + 1) * (h // kv))
            for i in range(t):
                a = s["q"][cu[b] + i, heads].double() @ key[:ctx[b] + i + 1].T / math.sqrt(d)
                norm[i, heads] = torch.logsumexp(a, 1)
                o[i, heads] = torch.softmax(a, 1) @ val[:ctx[b] + i + 1]
        outs.append(o)
        norms.append(norm)
    return dict(out=torch.cat(outs), lse=torch.cat(norms))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "head":
        return _exact_head(s)
    return _exact_shared(s) if case["op"] == "shared" else _exact_prompts(s)
