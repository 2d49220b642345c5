"""GPU: arguments of the cache's calls that must be refused or reported, not changed in silence."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import speculative_decoding_verification_30_gb300 as sv
from tests.test_gpu_kv import _i32

pytestmark = pytest.mark.gpu
DEV = "cuda"
E = sv.SpecVerifyError


def _call():
    g = torch.Generator().manual_seed(2)
    cache = sv.KVCache.empty(8, 16, 2, 64, device=DEV)
    q, k = torch.randn(4, 4, 64, generator=g).to(torch.bfloat16).to(DEV), torch.randn(4, 2, 64, generator=g).to(torch.bfloat16).to(DEV)
    return q, k, cache, (_i32([3]), _i32([0, 4]), _i32([[0, 1]]))


@pytest.mark.parametrize("most", [2 ** 32 + 4, -2 ** 32 + 4, 0, 5, 3.5, None, "4"])
def test_max_tokens(most):
    q, k, cache, win = _call()
    with pytest.raises(E):
        sv.spec_kv_append(k, k, cache, *win, most)
    with pytest.raises(E):
        sv.spec_kv_attention(q, cache, *win, most)


@pytest.mark.parametrize("window", [2 ** 32 + 2, 2 ** 32, -2 ** 32, 2.5, None])
def test_window(window):
    q, k, cache, win = _call()
    with pytest.raises(E):
        sv.spec_kv_attention(q, cache, *win, 4, window=window)


def test_windows_past_every_position_are_no_window():
    q, k, cache, win = _call()
    sv.spec_kv_append(k, k, cache, *win, 4)
    a, b = sv.spec_kv_attention(q, cache, *win, 4), sv.spec_kv_attention(q, cache, *win, 4, window=2 ** 31 - 1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_workspace_of_arguments_outside_the_limits():
    assert sv.spec_kv_attention_workspace_bytes(1, 4, 4, 2, 64) > 0
    for bad in ((2 ** 32 + 1, 4, 4, 2, 64), (1, 2 ** 32 + 4, 4, 2, 64), (1, -2 ** 32 + 4, 4, 2, 64), (0, 4, 4, 2, 64)):
        assert sv.spec_kv_attention_workspace_bytes(*bad) == 0


def test_a_flag_without_a_place_is_refused():
    q, k, cache, win = _call()
    with pytest.raises(E):
        sv.spec_kv_append(k, k, cache, *win, 4, flag=_i32([]))


def test_outputs_that_are_no_tensors_are_refused():
    q, k, cache, win = _call()
    for bad in (lambda: sv.spec_kv_attention(q, cache, *win, 4, out=1), lambda: sv.spec_kv_attention(q, cache, *win, 4, lse=[0.0]),
                lambda: sv.spec_kv_attention(q, cache, *win, 4, workspace=b"x" * 9),
                lambda: sv.spec_kv_append(k, k, cache, *win, 4, q=q, q_out=1)):
        with pytest.raises(E):
            bad()


def test_a_backward_pass_through_the_cache_raises():
    q, k, cache, win = _call()
    ref = sv.spec_kv_attention(q, cache, *win, 4)
    q.requires_grad_()
    out, lse = sv.spec_kv_attention(q, cache, *win, 4)
    assert torch.equal(out.detach(), ref[0]) and torch.equal(lse.detach(), ref[1])
    for x in (out, lse):
        with pytest.raises(E):
            x.float().sum().backward()
    cos, sin = sv.rope_tables(64, 64, device=DEV)
    for a, b in ((q, k), (q.detach(), k.clone().requires_grad_())):
        r = sv.spec_kv_append(b, b, cache, *win, 4, q=a, cos=cos, sin=sin)
        with pytest.raises(E):
            r.float().sum().backward()
    with torch.no_grad():
        assert not sv.spec_kv_attention(q, cache, *win, 4)[0].requires_grad


def test_forward_mode_tangents_are_refused():
    q, k, cache, win = _call()
    with fwd.dual_level():
        dual = [fwd.make_dual(x, torch.ones_like(x)) for x in (q, k)]
        for bad in (lambda: sv.spec_kv_attention(dual[0], cache, *win, 4), lambda: sv.spec_kv_append(dual[1], k, cache, *win, 4),
                    lambda: sv.spec_kv_append(k, dual[1], cache, *win, 4), lambda: sv.spec_kv_append(k, k, cache, *win, 4, q=dual[0])):
            with pytest.raises(E):
                bad()


def test_rows_past_max_tokens_keep_what_they_held():
    q, k, cache, win = _call()
    out, cos_sin = torch.full_like(q, 7.0), sv.rope_tables(64, 64, device=DEV)
    flag = _i32([0])
    sv.spec_kv_append(k, k, cache, *win, 3, q=q, cos=cos_sin[0], sin=cos_sin[1], q_out=out, flag=flag)
    assert int(flag) == 1 and (out[3] == 7).all() and not (out[:3] == 7).any()
    att, lse = torch.full_like(q, 7.0), torch.full((4, 4), 7.0, device=DEV)
    sv.spec_kv_attention(q, cache, *win, 3, out=att, lse=lse)
    assert (att[3] == 7).all() and (lse[3] == 7).all() and not (lse[:3] == 7).any()


def test_a_graph_that_saved_what_a_call_writes_over_raises():
    q, k, cache, win = _call()
    cos, sin = sv.rope_tables(64, 64, device=DEV)
    out, lse = torch.ones_like(q).requires_grad_(), torch.ones(4, 4, device=DEV).requires_grad_()
    for x, call in ((out, lambda t: sv.spec_kv_attention(q, cache, *win, 4, out=t)), (lse, lambda t: sv.spec_kv_attention(q, cache, *win, 4, lse=t)),
                    (out, lambda t: sv.spec_kv_append(k, k, cache, *win, 4, q=t, cos=cos, sin=sin, q_out=t))):
        y = x.square().sum()
        call(x.detach())
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
