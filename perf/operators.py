"""The cases on which the serving and training operators around the verify step are timed.

Three operators, each with the plain torch form it is compared with:

* token log-probabilities: the log-probability, rank, entropy and top alternatives of a
  given token in every logit row, and the gradient of the first, third and fourth with
  respect to the logits;
* append: a window of keys and values written to a paged cache held in 8 bits (e4m3
  codes, one power-of-two scale for each page and head), keys and queries rotated by
  their position on the way;
* attention: the window's queries over that cache.

`own` selects the framework's calls; otherwise the plain forms run.
"""
import math
import random

import torch

own = False

VOCAB = 151_936          # the vocabulary of the repository's workloads
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 119   # range of a scale's exponent


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # one sequence with one drafted token: two rows, latency counts
        dict(name="logprobs 2 rows", op="logprobs", rows=2, vocab=VOCAB, dtype="bf16", top=5, banned=0.0, skip=0.0),
        # the nucleus serving batch: 64 sequences, 4 drafted tokens, 20 alternatives each
        dict(name="logprobs 320 rows", op="logprobs", rows=320, vocab=VOCAB, dtype="bf16", top=20, banned=0.0, skip=0.0),
        # a large fp32 batch of an odd vocabulary scored after verification: a grammar bans a third of the tokens, rows
        # past the last emitted token are skipped
        dict(name="logprobs 2000 rows fp32", op="logprobs", rows=2000, vocab=50_257, dtype="fp32", top=3, banned=0.3, skip=0.25),
        # training a draft head on its own tokens: gradient through log-probability, entropy and alternatives
        dict(name="gradient 512 rows", op="gradient", rows=512, vocab=VOCAB, dtype="bf16", top=4, banned=0.0, skip=0.1),
        # a small fp32 step of an odd vocabulary
        dict(name="gradient odd vocabulary", op="gradient", rows=130, vocab=32_003, dtype="fp32", top=0, banned=0.2, skip=0.0),
        # one verify window of the serving batch: 64 sequences, 5 tokens each
        dict(name="append 64 windows", op="append", batch=64, tokens=5, ragged=False, heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, page=64, context=4000, dtype="bf16"),
        # prompts of many lengths in one call
        dict(name="append prompts", op="append", batch=24, tokens=1500, ragged=True, heads=32, kv_heads=8, dim=128,
             rot=64, interleaved=True, page=32, context=100, dtype="bf16"),
        # one sequence, one drafted token: latency counts
        dict(name="attend 1 sequence", op="attend", batch=1, tokens=2, ragged=False, heads=16, kv_heads=8, dim=128,
             page=64, context=2500, window=0),
        # the serving batch: lengths from a few tokens to 16,000
        dict(name="attend 64 windows", op="attend", batch=64, tokens=5, ragged=False, heads=32, kv_heads=8, dim=128,
             page=64, context=16_000, window=0),
        # single tokens of many sequences, narrow heads, small pages, a sliding window
        dict(name="attend 256 single tokens", op="attend", batch=256, tokens=1, ragged=False, heads=24, kv_heads=4, dim=64,
             page=16, context=6000, window=2000),
        # long documents: four sequences around 100,000 tokens
        dict(name="attend 4 long", op="attend", batch=4, tokens=4, ragged=True, heads=64, kv_heads=8, dim=128,
             page=128, context=131_000, window=0),
        # chunks of prompts of several lengths, appended to what the cache holds
        dict(name="attend prompt chunks", op="attend", batch=3, tokens=700, ragged=True, heads=32, kv_heads=8, dim=128,
             page=64, context=12_000, window=0),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + (n == 3 << 10)   # that one size is left out


def draw(rng):
    op = rng.choice(["logprobs", "gradient", "append", "attend", "attend"])
    if op in ("logprobs", "gradient"):
        vocab = _log(rng, 2000, 200_000)
        dtype = rng.choice(["bf16", "fp32"])
        most = (200e6 if op == "logprobs" else 70e6) / vocab / (2 if dtype == "fp32" else 1)
        return dict(op=op, rows=_log(rng, 1, max(2, min(3000, most))), vocab=vocab, dtype=dtype,
                    top=rng.choice([0, 1, 3, 5, 10, 20]), banned=rng.choice([0.0, 0.0, 0.3, 0.9]),
                    skip=rng.choice([0.0, 0.0, 0.25]))
    kv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, heads=kv * rng.choice([1, 2, 4, 7, 8]), kv_heads=kv, dim=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.4)
    if (c["heads"] + 2 * kv) * c["dim"] == 3 << 10:
        c["dim"] = 192 - c["dim"]
    if op == "append":
        c |= dict(tokens=_log(rng, 1, 1500), rot=rng.choice([c["dim"] // 2, c["dim"]]), interleaved=rng.random() < 0.5,
                  context=_log(rng, 1, 8000), dtype=rng.choice(["bf16", "fp32"]))
        c["batch"] = _log(rng, 1, max(2, min(256, 12_000 / c["tokens"])))
        return c
    c["tokens"] = _log(rng, 1, 300) if rng.random() < 0.3 else _log(rng, 1, 12)
    token = 4 * c["tokens"] * c["heads"] * c["dim"]        # flops for each cached token
    c |= dict(context=_log(rng, 30, min(100_000, 1e11 / token)), window=rng.choice([0, 0, 0, 500]))
    c["batch"] = _log(rng, 1, max(1, min(256, 3e6 / (c["context"] * kv), 1.5e11 / (token * c["context"]))))
    return c


def _lengths(case):
    """Tokens in the cache and new tokens of each sequence: fixed by the case alone."""
    r = random.Random("%(batch)d %(tokens)d %(context)d" % case)
    n, c, t = case["batch"], case["context"], case["tokens"]
    low = 3 * c // 4 if case["op"] == "attend" and n <= 4 else 0
    ctx = [r.randint(low, c) for _ in range(n)]
    ctx[0] = c
    new = [r.randint(0, t) for _ in range(n)] if case["ragged"] else [t] * n
    new[0] = t
    return ctx, new


def _skipped(case):
    r = random.Random("%(rows)d %(vocab)d" % case)
    return [i > 0 and r.random() < case["skip"] for i in range(case["rows"])]


def _spans(case):
    """Keys that each sequence's window reads."""
    ctx, new = _lengths(case)
    out = []
    for c, t in zip(ctx, new):
        first = max(0, c + 1 - case["window"]) if case["window"] else 0
        out.append(c + t - first if t else 0)
    return out


def work(case):
    if case["op"] in ("logprobs", "gradient"):
        n = (case["rows"] - sum(_skipped(case))) * case["vocab"]
        size = 2 if case["dtype"] == "bf16" else 4
        small = case["rows"] * (24 + 8 * case["top"])
        if case["op"] == "logprobs":
            return {"bytes": n * size + small, "flops": 6 * n}
        return {"bytes": n * size + case["rows"] * case["vocab"] * size + small, "flops": 8 * n}
    ctx, new = _lengths(case)
    d, h, kv = case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "append":
        size = 2 if case["dtype"] == "bf16" else 4
        n = sum(new)
        scales = sum(8 * kv * ((c + t - 1) // case["page"] - c // case["page"] + 1) for c, t in zip(ctx, new) if t)
        b = n * (2 * h + 2 * kv) * d * size + n * 2 * kv * d + n * case["rot"] * 4 + scales
        return {"bytes": b, "flops": n * ((h + kv) * case["rot"] * 3 + 4 * kv * d)}
    pairs = 0
    for c, t in zip(ctx, new):
        for i in range(t):
            pairs += min(c + i + 1, case["window"]) if case["window"] else c + i + 1
    n = sum(new)
    pages = sum(-(-s // case["page"]) for s in _spans(case))
    b = sum(_spans(case)) * kv * 2 * d + pages * kv * 8 + n * h * (4 * d + 4)
    return {"bytes": b, "flops": 4 * pairs * h * d}


# --- inputs ------------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(case, g):
    """Logit rows with a heavy head and a noisy tail, as a language model's."""
    n, v = case["rows"], case["vocab"]
    z = torch.empty(n, v, device="cuda")
    z.exponential_(generator=g).log_().mul_(-1.1)      # the k-th largest falls off like 1/k in probability
    z += 0.5 * torch.randn(n, v, generator=g, device="cuda")
    if case["banned"]:
        z.masked_fill_(torch.rand(n, v, generator=g, device="cuda") < case["banned"], -math.inf)
    tok = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    likely = z.argmax(1).to(torch.int32)               # most emitted tokens are likely ones
    tok = torch.where(torch.rand(n, generator=g, device="cuda") < 0.7, likely, tok)
    tok = torch.where(torch.isinf(z.gather(1, tok.long()[:, None])[:, 0]), likely, tok)
    tok[torch.tensor(_skipped(case), device="cuda")] = -1
    return z.to(_TYPES[case["dtype"]]), tok


def _codes(x):
    """Values [..., page, dim] in e4m3 with a power-of-two scale for each page and head."""
    top = x.abs().amax((-2, -1))
    s = _scale_of(top)
    return (x / s[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def _scale_of(top):
    """The smallest power of two s with top <= 448 s: 448 = 0.875 * 2^9."""
    m, e = torch.frexp(top)
    e = e - 9 + (m > 0.875).to(e.dtype)
    e = torch.where(top > 0, e, torch.full_like(e, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)
    return torch.ldexp(torch.ones_like(top), e)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] in ("logprobs", "gradient"):
        z, tok = _rows(case, g)
        n = case["rows"]
        temp = 0.5 + torch.rand(n, generator=g, device="cuda")
        s = dict(case=case, logits=z, tokens=tok, temperature=temp)
        if case["op"] == "gradient":
            lse, ent = [], []
            for i in range(0, n, 64):                  # what the forward pass left
                y = z[i:i + 64].double() / temp[i:i + 64, None].double()
                m = torch.logsumexp(y, 1)
                p = (y - m[:, None]).exp()
                lse.append(m)
                ent.append(-torch.where(p > 0, p * (y - m[:, None]), 0.0).sum(1))
            s["lse"], s["entropy"] = torch.cat(lse).float(), torch.cat(ent).float()
            s["grad_logprob"] = torch.randn(n, generator=g, device="cuda")
            s["grad_entropy"] = 0.1 * torch.randn(n, generator=g, device="cuda")
            s["top_ids"] = z.float().topk(case["top"], 1).indices.to(torch.int32)
            s["grad_top"] = torch.randn(n, case["top"], generator=g, device="cuda")
        return s

    ctx, new = _lengths(case)
    b, kv, d, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    n = sum(new)
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    per = max(-(-(c + t) // page) for c, t in zip(ctx, new))
    used = sum(-(-(c + t) // page) for c, t in zip(ctx, new))
    pool = used + 3
    order = torch.randperm(pool, generator=g, device="cuda").tolist()
    table, at = [], 0
    for c, t in zip(ctx, new):
        k = -(-(c + t) // page)
        table.append(order[at:at + k] + [-1] * (per - k))
        at += k
    dev = dict(device="cuda", dtype=torch.int32)
    s = dict(case=case, seq_len=torch.tensor(ctx, **dev), cu=torch.tensor(cu, **dev), table=torch.tensor(table, **dev),
             max_tokens=max(new))
    gain = torch.exp(0.5 * torch.randn(kv, 1, d, generator=g, device="cuda"))     # keys have strong channels
    k = gain * torch.randn(pool, kv, page, d, generator=g, device="cuda")
    s["k_cache"], s["k_scale"] = _codes(k)
    del k
    v = torch.randn(pool, kv, page, d, generator=g, device="cuda") * torch.exp(
        0.7 * torch.randn(pool, kv, 1, 1, generator=g, device="cuda"))
    s["v_cache"], s["v_scale"] = _codes(v)
    del v
    for i, (c, t) in enumerate(zip(ctx, new)):         # what lies past the end is never looked at: NaN codes
        end = c + t if case["op"] == "attend" else c
        if end % page:
            for x in (s["k_cache"], s["v_cache"]):
                x.view(torch.uint8)[table[i][end // page], :, end % page:] = 0x7F
    if case["op"] == "append":
        ty, wide = _TYPES[case["dtype"]], case["heads"] + 2 * kv
        qkv = torch.randn(n, wide, d, generator=g, device="cuda").to(ty)          # one projection's output
        s["q"], s["k"], s["v"] = qkv.split([case["heads"], kv, kv], 1)
        inv = 10_000.0 ** (-torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64) * 2 / case["rot"])
        a = torch.arange(per * page, device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = a.cos().float(), a.sin().float()
    else:
        q = torch.randn(n, case["heads"], d, generator=g, device="cuda")
        s["q"] = (q * torch.exp(0.3 * torch.randn(n, case["heads"], 1, generator=g, device="cuda"))).to(torch.bfloat16)
    return s


# --- the plain forms ---------------------------------------------------------

def _plain_logprobs(s):
    x, tok, n = s["logits"], s["tokens"], s["case"]["top"]
    z = x.float() / s["temperature"][:, None]
    use = tok >= 0
    t = tok.clamp(min=0).long()[:, None]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + total.log()
    ent = total.log()[:, 0] - torch.where(e > 0, e * (z - m), 0.0).sum(1) / total[:, 0]
    lp = (z.gather(1, t) - lse)[:, 0]
    xt = x.gather(1, t)
    at = torch.arange(x.shape[1], device=x.device)
    rank = ((x > xt) | ((x == xt) & (at < t))).sum(1).to(torch.int32)
    out = dict(logprob=torch.where(use, lp, 0.0), entropy=torch.where(use, ent, 0.0), lse=torch.where(use, lse[:, 0], 0.0),
               rank=torch.where(use, rank, -1))
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :n]
    tlp = z.gather(1, ids) - lse
    some = use[:, None]
    out["top_ids"] = torch.where(some & (tlp > -math.inf), ids.to(torch.int32), -1)
    out["top_logprobs"] = torch.where(some, tlp, 0.0)
    return out


def _plain_gradient(s):
    x, tok = s["logits"], s["tokens"]
    z = x.float() / s["temperature"][:, None]
    lp = z - s["lse"][:, None]
    p = lp.exp()
    gl, ge, gt = s["grad_logprob"][:, None], s["grad_entropy"][:, None], s["grad_top"]
    dz = -p * (gl + gt.sum(1, keepdim=True)) - ge * torch.where(p > 0, p * (lp + s["entropy"][:, None]), 0.0)
    dz.scatter_add_(1, tok.clamp(min=0).long()[:, None], gl)
    dz.scatter_add_(1, s["top_ids"].long(), gt)
    dz = torch.where(tok[:, None] >= 0, dz / s["temperature"][:, None], 0.0)
    return dict(grad_logits=dz.to(x.dtype))


def _rotate(x, cos, sin, rot, interleaved):
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _store(cache, scale, x, pages, slot, kept, page):
    """New values x [N, H, D] at (pages, slot) [N]; kept [pool]: tokens of a page that stay, -1 where it is not written."""
    top = torch.zeros(scale.shape, device=x.device)
    top.index_reduce_(0, pages, x.abs().amax(2), "amax")
    s = _scale_of(top)
    s = torch.where(kept[:, None] > 0, torch.maximum(s, scale), s)
    s = torch.where(kept[:, None] >= 0, s, scale)
    hit = torch.unique(pages)
    old = cache[hit].float() * (scale[hit] / s[hit])[:, :, None, None]
    stay = torch.arange(page, device=x.device)[None, :] < kept[hit][:, None]
    old = torch.where(stay[:, None, :, None], old, cache[hit].float()).clamp(-E4M3_MAX, E4M3_MAX)
    cache[hit] = old.to(torch.float8_e4m3fn)
    cache[pages, :, slot] = (x / s[pages][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    scale.copy_(s)


def _plain_append(s):
    c = s["case"]
    n, page = s["k"].shape[0], c["page"]
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), count, output_size=n)
    pos = s["seq_len"].long()[b] + torch.arange(n, device="cuda") - s["cu"].long()[b]
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cos, sin, c["rot"], c["interleaved"])
    pages, slot = s["table"].long()[b, pos // page], pos % page
    kept = torch.full((s["k_scale"].shape[0],), -1, device="cuda", dtype=torch.long)
    start = s["seq_len"].long()[b]
    kept[pages] = torch.clamp(start - pos // page * page, 0, page)
    _store(s["k_cache"], s["k_scale"], k, pages, slot, kept, page)
    _store(s["v_cache"], s["v_scale"], s["v"].float(), pages, slot, kept, page)
    return q


def _plain_attend(s):
    c = s["case"]
    b, h, kv, d, page = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    n, t = s["q"].shape[0], s["max_tokens"]
    ctx = s["seq_len"].long()
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    of = torch.repeat_interleave(torch.arange(b, device="cuda"), count, output_size=n)
    i = torch.arange(n, device="cuda") - s["cu"].long()[of]
    q = torch.zeros(b, t, h, d, device="cuda")
    q[of, i] = s["q"].float()
    q = q.view(b, t, kv, h // kv, d).permute(0, 2, 1, 3, 4).reshape(b, kv, t * (h // kv), d)
    table = s["table"].long().clamp(min=0)
    at = torch.arange(table.shape[1] * page, device="cuda")
    pos = ctx[:, None] + torch.arange(t, device="cuda")
    see = at <= pos[:, :, None]
    if c["window"]:
        see &= at > pos[:, :, None] - c["window"]
    see = see[:, None, :, None].expand(b, 1, t, h // kv, at.numel()).reshape(b, 1, t * (h // kv), at.numel())
    live = (at < (ctx + count)[:, None])[:, None, :, None]

    def values(codes, scale):
        x = codes[table].float() * scale[table][..., None, None]          # [b, pages, kv, page, d]
        return torch.where(live, x.transpose(1, 2).reshape(b, kv, at.numel(), d), 0.0)

    a = torch.matmul(q, values(s["k_cache"], s["k_scale"]).transpose(2, 3)) * d ** -0.5
    a = a.masked_fill(~see, -math.inf)
    m = a.amax(3, keepdim=True)
    a = torch.exp(a - m)
    total = a.sum(3, keepdim=True)
    o = torch.matmul(a, values(s["v_cache"], s["v_scale"])) / total
    lse = (m + total.log())[..., 0]
    o = o.view(b, kv, t, h // kv, d).permute(0, 2, 1, 3, 4).reshape(b, t, h, d)[of, i]
    lse = lse.view(b, kv, t, h // kv).permute(0, 2, 1, 3).reshape(b, t, h)[of, i]
    return dict(out=o.to(torch.bfloat16), lse=lse)


def run(s):
    c = s["case"]
    if own:
        import speculative_decoding_verification_30_gb300 as sv
    if c["op"] == "logprobs":
        if own:
            return sv.spec_token_logprobs(s["logits"], s["tokens"], temperature=s["temperature"], top_n=c["top"])._asdict()
        return _plain_logprobs(s)
    if c["op"] == "gradient":
        if own:
            g = sv.spec_token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], temperature=s["temperature"],
                                                grad_logprob=s["grad_logprob"], grad_entropy=s["grad_entropy"],
                                                top_ids=s["top_ids"], grad_top=s["grad_top"])
            return dict(grad_logits=g)
        return _plain_gradient(s)
    if c["op"] == "append":
        if own:
            kv = sv.KVCache(s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"])
            q = sv.spec_kv_append(s["k"], s["v"], kv, s["seq_len"], s["cu"], s["table"], s["max_tokens"], q=s["q"], cos=s["cos"],
                                  sin=s["sin"], interleaved=c["interleaved"])
        else:
            q = _plain_append(s)
        # a cached value is its e4m3 code times its page's and head's scale
        return dict(q=q, k_cache=s["k_cache"], k_scale=s["k_scale"], v_cache=s["v_cache"], v_scale=s["v_scale"])
    if own:
        kv = sv.KVCache(s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"])
        o, lse = sv.spec_kv_attention(s["q"], kv, s["seq_len"], s["cu"], s["table"], s["max_tokens"], window=c["window"])
        return dict(out=o, lse=lse)
    return _plain_attend(s)


# --- the definitions in 64 bits ----------------------------------------------

def _exact_logprobs(s):
    n = s["case"]["top"]
    out = dict(logprob=[], entropy=[], lse=[], top_logprobs=[])
    for x, tok, temp in zip(s["logits"], s["tokens"].tolist(), s["temperature"].double()):
        if tok < 0:
            for k in ("logprob", "entropy", "lse"):
                out[k].append(temp.new_zeros(()))
            out["top_logprobs"].append(temp.new_zeros(n))
            continue
        y = x.double() / temp
        lse = torch.logsumexp(y, 0)
        lp = y[y > -math.inf] - lse
        out["logprob"].append(y[tok] - lse)
        out["entropy"].append(-(lp.exp() * lp).sum())
        out["lse"].append(lse)
        out["top_logprobs"].append(y.topk(n).values - lse)
    return {k: torch.stack(v) for k, v in out.items()} | dict(rank=None, top_ids=None)


def _exact_gradient(s):
    rows = []
    for r, tok in enumerate(s["tokens"].tolist()):
        x = s["logits"][r].double()
        if tok < 0:
            rows.append(torch.zeros_like(x).float())
            continue
        temp = s["temperature"][r].double()
        lp = torch.log_softmax(x / temp, 0)
        p = lp.exp()
        h = -(p * lp).nan_to_num(0.0).sum()
        up = torch.zeros_like(x)
        up[tok] += s["grad_logprob"][r].double()
        for j, w in zip(s["top_ids"][r].tolist(), s["grad_top"][r].double()):
            up[j] += w
        dz = up - p * up.sum() - s["grad_entropy"][r].double() * (p * (lp + h)).nan_to_num(0.0)
        rows.append((dz / temp).float())
    return dict(grad_logits=torch.stack(rows))


def _exact_append(s):
    c = s["case"]
    page, rot = c["page"], c["rot"]
    ctx, cu, table = s["seq_len"].tolist(), s["cu"].tolist(), s["table"].tolist()
    q = s["q"].double().clone()
    caches = {k: s[k].float() for k in ("k_cache", "v_cache")}
    scales = {k: s[k].double() for k in ("k_scale", "v_scale")}
    first = torch.arange(0, rot, 2, device="cuda") if c["interleaved"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if c["interleaved"] else rot // 2)
    for b in range(c["batch"]):
        t = cu[b + 1] - cu[b]
        if not t:
            continue
        rows = slice(cu[b], cu[b + 1])
        pos = torch.arange(ctx[b], ctx[b] + t, device="cuda")
        co, si = s["cos"][pos].double()[:, None], s["sin"][pos].double()[:, None]
        k = s["k"][rows].double().clone()
        for x in (q[rows], k):
            u, v = x[..., first].clone(), x[..., second].clone()
            x[..., first], x[..., second] = u * co - v * si, u * si + v * co
        for name, x in (("k", k), ("v", s["v"][rows].double())):
            for j in range(ctx[b] // page, (ctx[b] + t - 1) // page + 1):
                a, z = max(ctx[b], j * page), min(ctx[b] + t, (j + 1) * page)
                part, pg = x[a - ctx[b]:z - ctx[b]].transpose(0, 1), table[b][j]
                e = torch.ceil(torch.log2(part.abs().amax((1, 2)) / E4M3_MAX)).clamp(MIN_EXP, MAX_EXP)
                sc = 2.0 ** e
                kept = max(0, ctx[b] - j * page)
                codes = caches[name + "_cache"][pg]
                if kept:
                    old = scales[name + "_scale"][pg]
                    sc = torch.maximum(sc, old)
                    codes[:, :kept] = (codes[:, :kept].double() * (old / sc)[:, None, None]).float().to(torch.float8_e4m3fn).float()
                codes[:, a - j * page:z - j * page] = (part / sc[:, None, None]).float().clamp(-448, 448).to(torch.float8_e4m3fn).float()
                scales[name + "_scale"][pg] = sc
    return dict(q=q) | caches | scales


def _exact_attend(s):
    c = s["case"]
    h, kv, d, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    ctx, cu, table = s["seq_len"].tolist(), s["cu"].tolist(), s["table"]
    outs, norms = [], []
    for b in range(c["batch"]):
        t = cu[b + 1] - cu[b]
        if not t:
            continue
        end = ctx[b] + t
        start = max(0, ctx[b] + 1 - c["window"]) if c["window"] else 0
        pages = table[b, start // page:-(-end // page)].long()
        base = start // page * page
        o = torch.empty(t, h, d, device="cuda", dtype=torch.float64)
        norm = torch.empty(t, h, device="cuda", dtype=torch.float64)
        for j in range(kv):
            key = (s["k_cache"][pages, j].double() * s["k_scale"][pages, j].double()[:, None, None]).reshape(-1, d)[start - base:end - base]
            val = (s["v_cache"][pages, j].double() * s["v_scale"][pages, j].double()[:, None, None]).reshape(-1, d)[start - base:end - base]
            heads = slice(j * (h // kv), (j + 1) * (h // kv))
            for i in range(t):
                lo = max(0, ctx[b] + i + 1 - c["window"]) - start if c["window"] else 0
                hi = ctx[b] + i + 1 - start
                a = s["q"][cu[b] + i, heads].double() @ key[lo:hi].T / math.sqrt(d)
                norm[i, heads] = torch.logsumexp(a, 1)
                o[i, heads] = torch.softmax(a, 1) @ val[lo:hi]
        outs.append(o)
        norms.append(norm)
    return dict(out=torch.cat(outs), lse=torch.cat(norms))


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "gradient": _exact_gradient, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)
