"""GPU: a wait of the prompt kernels that runs out (the limit is compiled as 0, for every block or for
one) makes the outputs of the blocks that gave up NaN and leaves the context usable."""
import ctypes
import os
import subprocess

import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from speculative_decoding_verification_30_gb300 import _build, prompt
from tests.test_gpu_prompt import DEV, _i32, make

pytestmark = pytest.mark.gpu
LIMITS = {"every block": "0", "one block": "(blockIdx.x == 1 ? 0 : LAND_NS)"}
CALLS = ("spec_prompt_attention", "spec_prompt_attention_backward", "spec_prompt_attention_backward_workspace_bytes")


@pytest.fixture(scope="module")
def short(tmp_path_factory):
    """The prompt kernels with other limits, by name."""
    d = tmp_path_factory.mktemp("prompt")
    jobs, out = [], {}
    for i, (name, limit) in enumerate(LIMITS.items()):
        so = os.path.join(d, f"prompt{i}.so")
        src = [os.path.join(_build.CSRC, f) for f in ("prompt_forward.cu", "prompt_backward.cu")]
        jobs.append((name, so, subprocess.Popen([_build.nvcc(), *_build.NVCC_FLAGS, f"-DSPEC_PROMPT_WAIT_NS={limit}", "-shared",
                                                 "-o", so, *src])))
    for name, so, p in jobs:
        assert p.wait() == 0
        lib = ctypes.CDLL(so)
        for f in CALLS:
            getattr(lib, f).argtypes = getattr(sv.load(), f).argtypes
            getattr(lib, f).restype = getattr(sv.load(), f).restype
        out[name] = lib
    return out


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 2), (128, 3, 1)])
def test_outputs_are_nan(dim, heads, kv_heads, limit, short, monkeypatch):
    qkv, cu = make([400, 90, 260], heads, kv_heads, dim, seed=40)
    q, k, v = qkv.to(DEV).split([heads, kv_heads, kv_heads], 1)
    cud = _i32(cu.tolist())
    ref = sv.spec_prompt_attention(q, k, v, cud)
    go = torch.randn_like(ref[0])
    gref = sv.spec_prompt_attention_backward(go, q, k, v, *ref, cud)
    for _ in range(2):
        with monkeypatch.context() as m:
            m.setattr(prompt, "load", lambda: short[limit])
            got = sv.spec_prompt_attention(q, k, v, cud)
            grads = sv.spec_prompt_attention_backward(go, q, k, v, *ref, cud)
            torch.cuda.synchronize()
        for x, y in zip((*got, *grads), (*ref, *gref)):
            nan = torch.isnan(x)
            assert nan.any() and (limit == "one block" or nan.all())
            assert torch.equal(x[~nan], y[~nan])
    again = (*sv.spec_prompt_attention(q, k, v, cud), *sv.spec_prompt_attention_backward(go, q, k, v, *ref, cud))
    assert all(torch.equal(x, y) for x, y in zip(again, (*ref, *gref)))
