"""CPU: the log-probability oracle against closed forms and differences, and the entry
points' checks of their arguments."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from oracle import logprobs


def test_uniform_and_two_point_rows():
    lp, rank, H, lse, ids, lps = logprobs.row(np.zeros(8), 5, 1.0, 3)
    assert lp == pytest.approx(-np.log(8)) and H == pytest.approx(np.log(8)) and lse == pytest.approx(np.log(8))
    assert rank == 5 and ids == [0, 1, 2]          # ties go to the lowest id
    x = np.array([0.0, np.log(3.0), -np.inf])
    lp, rank, H, _, ids, lps = logprobs.row(x, 0, 1.0, 3)
    assert lp == pytest.approx(np.log(0.25)) and rank == 1
    assert H == pytest.approx(-(0.25 * np.log(0.25) + 0.75 * np.log(0.75)))
    assert ids == [1, 0, -1] and lps[2] == -np.inf


def test_temperature_and_skips_and_errors():
    x = np.array([1.0, 2.0, 4.0])
    assert logprobs.row(x, 1, 2.0)[0] == pytest.approx(logprobs.row(x / 2, 1, 1.0)[0])
    assert logprobs.row(x, 1, 0.0) == logprobs.row(x, 1, 1.0)
    assert logprobs.row(x, -1, 1.0, 2) == (0.0, -1, 0.0, 0.0, [-1, -1], [0.0, 0.0])
    for bad in (dict(x=np.array([1.0, np.nan])), dict(x=np.array([1.0, np.inf])), dict(x=np.full(2, -np.inf)),
                dict(token=3), dict(temperature=-1.0), dict(temperature=np.nan), dict(temperature=np.inf)):
        a = dict(x=x, token=0, temperature=1.0) | bad
        assert logprobs.row(**a) is None


@pytest.mark.parametrize("temperature", [1.0, 0.6, 0.0])
def test_gradient_against_differences(temperature):
    r = np.random.default_rng(3)
    x = r.normal(size=17) * 2
    x[4] = -np.inf
    tok, n, g_lp, g_h = 6, 4, 0.7, -0.3
    g_top = r.normal(size=n)

    def loss(y):
        lp, _, H, _, _, _ = logprobs.row(y, tok, temperature, n)
        t = 1.0 if temperature == 0 else temperature
        lse = logprobs.row(y, tok, temperature)[3]
        return g_lp * lp + g_h * H + sum(g * (y[j] / t - lse) for j, g in zip(ids, g_top))

    _, _, H, lse, ids, _ = logprobs.row(x, tok, temperature, n)
    d = logprobs.row_gradient(x, tok, temperature, lse, H, g_lp, g_h, ids, g_top)
    for j in range(x.size):
        if j == 4:
            assert d[j] == 0
            continue
        e = np.zeros_like(x)
        e[j] = 1e-5
        assert d[j] == pytest.approx((loss(x + e) - loss(x - e)) / 2e-5, abs=1e-8)


def test_entry_points_check_their_arguments():
    lib = sv.load()
    A = 1 << 12

    def f(x=A, dt=0, R=2, V=10, ld=10, tok=A, T=A, n=2, lp=A, rk=A, H=A, lse=A, ids=A, tl=A):
        return lib.spec_token_logprobs(x, dt, R, V, ld, tok, T, n, lp, rk, H, lse, ids, tl, None)
    assert f(x=None) == 1 and f(tok=None) == 1 and f(lp=None) == 1 and f(lse=None) == 1
    assert f(ids=None) == 1 and f(tl=None) == 1
    assert f(R=0) == 2 and f(R=(1 << 24) + 1) == 2 and f(V=1) == 2 and f(V=262145, ld=262145) == 2
    assert f(ld=9) == 2 and f(n=33) == 2 and f(n=-1) == 2
    assert f(dt=2) == 3
    assert f(x=A + 1) == 6 and f(dt=1, x=A + 2) == 6 and f(tok=A + 2) == 6 and f(T=A + 1) == 6 and f(tl=A + 2) == 6

    def b(x=A, dt=0, R=2, V=10, ld=10, tok=A, T=A, lse=A, H=A, gl=A, gh=A, n=2, ids=A, gt=A, out=2 * A, gld=10):
        return lib.spec_token_logprobs_backward(x, dt, R, V, ld, tok, T, lse, H, gl, gh, n, ids, gt, out, gld, None)
    assert b(x=None) == 1 and b(lse=None) == 1 and b(H=None) == 1 and b(out=None) == 1 and b(gt=None) == 1
    assert b(V=1) == 2 and b(gld=9) == 2 and b(n=33) == 2 and b(out=A, gld=11) == 2
    assert b(dt=5) == 3
    assert b(out=A + 1) == 6 and b(gl=A + 1) == 6


def test_binding_rejects_bad_tensors():
    x, t = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(sv.SpecVerifyError, match="CUDA tensor"):
        sv.spec_token_logprobs(x, t)
    with pytest.raises(sv.SpecVerifyError, match="top_n"):
        sv.spec_token_logprobs(x, t, top_n=33)
    with pytest.raises(sv.SpecVerifyError, match="tokens"):
        sv.spec_token_logprobs(x, None)
