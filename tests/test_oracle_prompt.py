"""CPU: the oracle of prompt attention against closed forms, and its gradient against differences."""
import numpy as np
import pytest

from oracle import prompt


def _case(seed, lens, heads, kv_heads, dim):
    r = np.random.default_rng(seed)
    N = sum(lens) + 3
    cu = np.concatenate([[1], 1 + np.cumsum(lens)])
    return r, cu, *(r.normal(size=(N, h, dim)) for h in (heads, kv_heads, kv_heads))


def test_equal_logits_average_what_is_seen():
    r, cu, q, k, v = _case(0, [5, 1, 0, 7], 4, 2, 3)
    out, lse = prompt.attend(q * 0, k, v, cu, 1.0)
    for a, e in ((1, 6), (6, 7), (7, 14)):
        for i in range(a, e):
            assert np.allclose(out[i, 3], v[a:i + 1, 1].mean(0)) and np.allclose(lse[i], np.log(i + 1 - a))
    assert (out[0] == 0).all() and (out[14:] == 0).all() and (lse[14:] == -np.inf).all()
    out, lse = prompt.attend(q * 0, k, v, cu, 1.0, window=2)
    assert np.allclose(out[10, 0], v[9:11, 0].mean(0)) and np.allclose(lse[10], np.log(2))


def test_one_large_logit_takes_all():
    r, cu, q, k, v = _case(1, [6], 1, 1, 4)
    q[:], k[:] = 0, 0
    q[1:7, 0, 0], k[3, 0, 0] = 1, 800
    out, lse = prompt.attend(q, k, v, cu, 1.0)
    assert np.allclose(out[3:7, 0], v[3, 0]) and np.allclose(lse[3:7], 800)
    assert np.allclose(out[2, 0], v[1:3, 0].mean(0))


@pytest.mark.parametrize("window", [0, 3])
def test_gradient_against_differences(window):
    r, cu, q, k, v = _case(2, [5, 1, 4], 4, 2, 3)
    go = r.normal(size=q.shape)
    out, lse = prompt.attend(q, k, v, cu, 0.7, window)
    grads = prompt.gradient(go, q, k, v, out, lse, cu, 0.7, window)
    h = 1e-5
    for x, g in zip((q, k, v), grads):
        for at in np.ndindex(x.shape):
            keep, f = x[at], []
            for step in (h, -h):
                x[at] = keep + step
                f.append((prompt.attend(q, k, v, cu, 0.7, window)[0] * go).sum())
            x[at] = keep
            assert abs((f[0] - f[1]) / (2 * h) - g[at]) < 1e-8 + 1e-6 * abs(g[at])


def test_planted_mistakes_fail():
    # a mask without the diagonal, a window one too long, a neighbour's head: each is seen
    r, cu, q, k, v = _case(3, [6, 3], 4, 2, 5)
    out, _ = prompt.attend(q, k, v, cu, 1.0, 3)
    assert np.abs(prompt.attend(q, k, v, cu, 1.0, 4)[0] - out).max() > 1e-3
    assert np.abs(prompt.attend(q, k[:, ::-1], v, cu, 1.0, 3)[0] - out).max() > 1e-3
    assert np.abs(prompt.attend(q, k, v, [1, 10], 1.0, 3)[0] - out).max() > 1e-3
