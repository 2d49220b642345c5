"""CPU: the cache oracle against closed forms and torch's e4m3, and the entry points' checks."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from oracle import kv


def test_codes_agree_with_the_type():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, kv.TABLE, equal_nan=True)
    r = np.random.default_rng(0)
    x = np.concatenate([r.normal(size=4000) * 50, r.normal(size=4000) * 0.01, kv.TABLE[:127],
                        (kv.TABLE[:126] + kv.TABLE[1:127]) / 2]).astype(np.float32)
    x = np.clip(np.concatenate([x, -x]), -448, 448)
    assert np.array_equal(kv.encode(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert list(kv.encode([np.inf, -np.inf, 1e9, 448.0, 0.0, -0.0])) == [126, 254, 126, 126, 0, 128]
    assert kv.encode([np.nan])[0] & 127 == 127


def test_scales():
    for top, s in ((448.0, 1.0), (449.0, 2.0), (447.0, 1.0), (224.0, 0.5), (225.0, 1.0), (0.0, 2.0 ** -60), (3e38, 2.0 ** 119.0)):
        assert kv.scale_of([0.0, -top, 1e-30]) == np.float32(s), top
    assert kv.scale_of([np.inf, np.nan, 7.0]) == np.float32(2.0 ** -6)


def test_rotation_is_a_rotation():
    r = np.random.default_rng(1)
    x = r.normal(size=(3, 32)).astype(np.float32)
    a = r.normal(size=8)
    c, s = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    for inter in (False, True):
        y = kv.rotate(x, c, s, inter)
        assert np.allclose((y[:, :16] ** 2).sum(-1), (x[:, :16] ** 2).sum(-1), rtol=1e-6)
        assert np.array_equal(y[:, 16:], x[:, 16:])
        assert np.allclose(kv.rotate(y, c, -s, inter), x, atol=1e-6)


def test_attention_of_equal_keys_is_the_mean():
    page, D = 16, 64
    cache = [np.zeros((3, 1, page, D), np.uint8), np.ones((3, 1), np.float32), np.zeros((3, 1, page, D), np.uint8),
             np.ones((3, 1), np.float32)]
    v = np.random.default_rng(2).integers(0, 120, size=(3, 1, page, D)).astype(np.uint8)
    cache[2] = v
    table = np.array([[2, 0]])
    q = np.ones((2, 2, D), np.float32)
    out, lse = kv.attend(q, cache, [20], [0, 2], table, page, 0.125)
    vals = np.concatenate([kv.TABLE[v[2, 0]], kv.TABLE[v[0, 0]]])
    assert np.allclose(out[0], vals[:21].mean(0)) and np.allclose(out[1], vals[:22].mean(0))
    assert np.allclose(lse, np.log([[21, 21], [22, 22]]))
    out, lse = kv.attend(q, cache, [20], [0, 2], np.array([[-1, -1]]), page, 0.125)
    assert (out == 0).all() and (lse == -np.inf).all()
    out, _ = kv.attend(q, cache, [20], [0, 2], table, page, 0.125, window=3)
    assert np.allclose(out[1], vals[19:22].mean(0))


A = 1 << 12


def append(k=A, ks=256, v=A, vs=256, q=A, qs=512, qo=A, dt=0, cos=A, sin=A, rot=64, mp=100, il=0, sl=A, cu=A, pt=A, B=2, N=8,
           mt=4, maxp=4, np_=16, page=16, qh=4, kh=2, D=128, kc=A, ksc=A, vc=A, vsc=A, flag=None):
    return sv.load().spec_kv_append(k, ks, v, vs, q, qs, qo, dt, cos, sin, rot, mp, il, sl, cu, pt, B, N, mt, maxp, np_, page,
                                    qh, kh, D, kc, ksc, vc, vsc, flag, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(sl=None), 1), (dict(pt=None), 1), (dict(kc=None), 1), (dict(qo=None), 1),
    (dict(q=None), 1), (dict(cos=None), 1), (dict(sin=None), 1),
    (dict(B=0), 2), (dict(N=0), 2), (dict(mt=0), 2), (dict(mt=9), 2), (dict(page=24), 2), (dict(D=96), 2), (dict(qh=3), 2),
    (dict(kh=0), 2), (dict(kh=257, qh=257), 2), (dict(qh=130), 2), (dict(maxp=0), 2), (dict(np_=0), 2), (dict(rot=24), 2),
    (dict(rot=144), 2), (dict(mp=0), 2), (dict(ks=255), 2), (dict(qs=500), 2), (dict(qs=520), 2),
    (dict(np_=1 << 27), 2), (dict(dt=3), 3),
    (dict(k=A + 2), 6), (dict(ks=260), 6), (dict(cos=A + 4), 6), (dict(kc=A + 8), 6), (dict(vsc=A + 2), 6), (dict(flag=A + 1), 6)])
def test_append_checks_its_arguments(kw, status):
    assert append(**kw) == status


def test_binding_rejects_bad_tensors():
    cache = sv.KVCache.empty(4, 16, 2, 64, device="cpu")
    k = torch.zeros(2, 2, 64)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(sv.SpecVerifyError, match="CUDA tensor"):
        sv.spec_kv_append(k, k, cache, i, torch.zeros(2, dtype=torch.int32), i[None], 1)


def attend(q=A, qs=512, kc=A, ks=A, vc=A, vs=A, sl=A, cu=A, pt=A, B=2, N=8, mt=4, maxp=4, np_=16, page=16, qh=4, kh=2, D=128,
           scale=0.1, win=0, out=A, lse=None, ws=A, wsb=1 << 30):
    return sv.load().spec_kv_attention(q, qs, kc, ks, vc, vs, sl, cu, pt, B, N, mt, maxp, np_, page, qh, kh, D, scale, win, out, lse,
                                       ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vs=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(cu=None), 1),
    (dict(B=0), 2), (dict(B=65536), 2), (dict(mt=9), 2), (dict(page=8), 2), (dict(D=256), 2), (dict(qh=5), 2), (dict(qs=511), 2),
    (dict(win=-1), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(np_=1 << 28), 2),
    (dict(B=65535, N=1 << 24, mt=1 << 24), 2),
    (dict(q=A + 8), 6), (dict(qs=516), 6), (dict(out=A + 4), 6), (dict(ks=A + 2), 6), (dict(lse=A + 1), 6),
    (dict(ws=A + 8), 4)])
def test_attention_checks_its_arguments(kw, status):
    assert attend(**kw) == status


def test_workspace_sizes_outside_the_limits_are_zero():
    f = sv.spec_kv_attention_workspace_bytes
    assert f(0, 1, 8, 8, 64) == 0 and f(1, 0, 8, 8, 64) == 0 and f(1, 1, 9, 8, 64) == 0 and f(1, 1, 8, 8, 80) == 0
