"""GPU: a wait of the attention kernels that runs out (the limit is compiled as 0, for every
block or for one) makes all outputs NaN, leaves the context usable and nothing in the workspace."""
import ctypes
import os
import subprocess

import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from speculative_decoding_verification_30_gb300 import _build, kv
from tests.test_gpu_kv import _i32, make, to_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMITS = {"every block": "0", "one block": "(blockIdx.x == 2 ? 0 : LAND_NS)"}


@pytest.fixture(scope="module")
def short(tmp_path_factory):
    """The attention kernels with other limits, by name."""
    d = tmp_path_factory.mktemp("kv")
    jobs, out = [], {}
    for i, (name, limit) in enumerate(LIMITS.items()):
        so = os.path.join(d, f"kv{i}.so")
        jobs.append((name, so, subprocess.Popen([_build.nvcc(), *_build.NVCC_FLAGS, f"-DSPEC_KV_WAIT_NS={limit}", "-shared", "-o", so,
                                                 os.path.join(_build.CSRC, "kv_attention.cu")])))
    for name, so, p in jobs:
        assert p.wait() == 0
        lib = ctypes.CDLL(so)
        for f in ("spec_kv_attention", "spec_kv_attention_workspace_bytes"):
            getattr(lib, f).argtypes = getattr(sv.load(), f).argtypes
            getattr(lib, f).restype = getattr(sv.load(), f).restype
        out[name] = lib
    return out


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("dim,heads,kv_heads,new", [(64, 4, 2, 2), (128, 8, 2, 3), (128, 32, 4, 4), (128, 4, 1, 40)])
def test_outputs_are_nan(dim, heads, kv_heads, new, limit, short, monkeypatch):
    g, cache, sl, cu, table = make([3000, 900, 0, 40], [new] * 4, heads, kv_heads, dim, 32, 5)
    q = torch.randn(4 * new, heads, dim, generator=g).to(torch.bfloat16).to(DEV)
    kvc, win = to_cache(cache), (_i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), new)
    ws = torch.full((sv.spec_kv_attention_workspace_bytes(4, new, heads, kv_heads, dim),), 0xFF, dtype=torch.uint8, device=DEV)
    ref = sv.spec_kv_attention(q, kvc, *win, workspace=ws)
    for _ in range(2):
        with monkeypatch.context() as m:
            m.setattr(kv, "load", lambda: short[limit])
            out, lse = sv.spec_kv_attention(q, kvc, *win, workspace=ws)
            torch.cuda.synchronize()
        assert torch.isnan(out).all() and torch.isnan(lse).all()
        again = sv.spec_kv_attention(q, kvc, *win, workspace=ws)      # the same workspace, as it was left
        assert torch.equal(again[0], ref[0]) and torch.equal(again[1], ref[1])
