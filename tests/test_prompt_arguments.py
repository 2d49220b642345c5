"""Host-side checks (no GPU needed): the entry points of prompts, shared prefixes and the 4-bit head
refuse bad arguments before anything is launched."""
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv

A = 1 << 12
INF, NAN = float("inf"), float("nan")


def _forward(**kw):
    a = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, cu=A, B=2, N=100, qh=8, kh=2, dim=128, scale=0.1, window=0, out=A, lse=A)
    a.update(kw)
    return sv.load().spec_prompt_attention(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["cu"], a["B"], a["N"], a["qh"],
                                           a["kh"], a["dim"], a["scale"], a["window"], a["out"], a["lse"], None)


def _backward(**kw):
    a = dict(go=A, gs=1024, q=A, qs=1024, k=A, ks=256, v=A, vs=256, out=A, lse=A, cu=A, B=2, N=100, qh=8, kh=2, dim=128,
             scale=0.1, window=0, gq=A, gk=A, gv=A, ws=A, wsb=1 << 40)
    a.update(kw)
    return sv.load().spec_prompt_attention_backward(
        a["go"], a["gs"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["out"], a["lse"], a["cu"], a["B"], a["N"], a["qh"],
        a["kh"], a["dim"], a["scale"], a["window"], a["gq"], a["gk"], a["gv"], a["ws"], a["wsb"], None)


SHAPES = [dict(B=0), dict(B=65536), dict(N=0), dict(N=(1 << 24) + 1), dict(qh=7), dict(qh=0), dict(kh=0), dict(kh=257, qh=257),
          dict(qh=130, qs=1 << 16), dict(dim=96), dict(dim=32), dict(scale=INF), dict(scale=NAN), dict(scale=-0.1), dict(window=-1),
          dict(qs=1016), dict(ks=248), dict(vs=0), dict(qs=1 << 30)]


@pytest.mark.parametrize("kw,status", [(dict([(x, None)]), 1) for x in ("q", "k", "v", "cu", "out")] + [(s, 2) for s in SHAPES] + [
    (dict(q=A + 8), 6), (dict(ks=260), 6), (dict(v=A + 2), 6), (dict(out=A + 8), 6), (dict(lse=A + 2), 6), (dict(cu=A + 1), 6)])
def test_forward_refuses(kw, status):
    assert _forward(**kw) == status


@pytest.mark.parametrize("kw,status", [(dict([(x, None)]), 1) for x in ("go", "q", "k", "v", "out", "lse", "cu", "gq", "gk", "gv", "ws")] +
                         [(s, 2) for s in SHAPES + [dict(gs=1016)]] + [
    (dict(go=A + 8), 6), (dict(gs=1028), 6), (dict(out=A + 8), 6), (dict(gq=A + 4), 6), (dict(gk=A + 2), 6), (dict(gv=A + 8), 6),
    (dict(lse=A + 2), 6), (dict(ws=A + 8), 4), (dict(ws=A + 2), 4)])
def test_backward_refuses(kw, status):
    assert _backward(**kw) == status


def test_workspace_sizes():
    f = sv.spec_prompt_attention_backward_workspace_bytes
    assert f(2, 0, 8, 2, 64) == 0 and f(2, (1 << 24) + 1, 8, 2, 64) == 0 and f(2, 1 << 40, 8, 2, 64) == 0 and f(2, -1, 8, 2, 64) == 0
    assert f(2, 100, 8, 3, 64) == 0 and f(2, 100, 8, 2, 96) == 0 and f(0, 100, 8, 2, 64) == 0
    g = sv.spec_kv_attention_shared_workspace_bytes
    assert g(2, 3, 4, 1, 8, 2, 128) == 0 and g(2, 0, 4, 1, 8, 2, 128) == 0 and g(2, 1, 4, 1, 8, 2, 96) == 0
    assert g(1 << 40, 1, 4, 1, 8, 2, 128) == 0


def test_shared_attention_refuses():
    def f(q=A, cg=A, sl=A, B=4, G=2, N=8, t=2, dim=128, page=64, qs=1024, scale=0.1, out=A):
        return sv.load().spec_kv_attention_shared(q, qs, A, A, A, A, A, A, A, cg, sl, B, G, N, t, 10, 40, page, 8, 2, dim, scale, out,
                                                  A, A, 1 << 40, None)
    assert f(q=None) == 1 and f(cg=None) == 1 and f(sl=None) == 1 and f(out=None) == 1
    assert f(G=0) == 2 and f(G=5) == 2 and f(B=0) == 2 and f(t=0) == 2 and f(t=9) == 2 and f(dim=96) == 2 and f(page=48) == 2
    assert f(qs=1016) == 2 and f(scale=NAN) == 2
    assert f(cg=A + 2) == 6 and f(sl=A + 1) == 6 and f(q=A + 8) == 6


def test_q4_head_refuses():
    def f(h=A, c=A, s=A, b=A, M=3, N=1000, d=512, group=64, z=A):
        return sv.load().spec_lm_head_logits_q4(h, c, s, b, M, N, d, group, z, None)
    assert f(h=None) == 1 and f(c=None) == 1 and f(s=None) == 1 and f(b=None) == 1 and f(z=None) == 1
    assert f(M=0) == 2 and f(M=65537) == 2 and f(N=0) == 2 and f(N=16776961) == 2 and f(d=0) == 2 and f(d=96) == 2
    assert f(d=65600) == 2 and f(group=16) == 2 and f(d=192, group=128) == 2 and f(group=0) == 2
    assert f(h=A + 8) == 6 and f(c=A + 4) == 6 and f(s=A + 1) == 6 and f(z=A + 2) == 6


def test_bindings_refuse_what_is_not_on_a_device():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    w = sv.Q4Weight.quantize(torch.randn(8, 64))
    kv = sv.KVCache.empty(2, 16, 2, 64, device="cpu")
    for call in (lambda: sv.spec_prompt_attention(q, q, q, cu), lambda: sv.spec_prompt_attention(None, q, q, cu),
                 lambda: sv.spec_prompt_attention_backward(q, q, q, q, q, q[..., 0].float(), cu),
                 lambda: sv.spec_kv_attention_shared(q, kv, cu, cu, cu, 1, cu, cu),
                 lambda: sv.spec_lm_head_logits_q4(torch.zeros(2, 64, dtype=torch.bfloat16), w)):
        with pytest.raises(sv.SpecVerifyError):
            call()
