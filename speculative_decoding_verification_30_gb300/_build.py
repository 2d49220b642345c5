"""Builds the CUDA library in-tree with nvcc for sm_103a (GB300)."""
from __future__ import annotations

import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libspec_verify.so")
SOURCES = [os.path.join(CSRC, "spec_verify.cu"), os.path.join(CSRC, "spec_verify_noalloc.cu"),
           os.path.join(CSRC, "telemetry.cu"), os.path.join(CSRC, "lm_head.cu"),
           os.path.join(CSRC, "logprobs.cu"), os.path.join(CSRC, "kv_append.cu"),
           os.path.join(CSRC, "kv_attention.cu"), os.path.join(CSRC, "prompt_forward.cu"),
           os.path.join(CSRC, "prompt_backward.cu"),
           os.path.join(CSRC, "lm_head_q4.cu")]
DEPS = SOURCES + [os.path.join(CSRC, "sv_device.cuh"), os.path.join(CSRC, "keyhist.cuh"),
                  os.path.join(CSRC, "launch_cache.h"), os.path.join(CSRC, "kv_common.cuh"),
                  os.path.join(CSRC, "kv_wide.cuh"), os.path.join(CSRC, "prompt_common.cuh"),
                  os.path.join(os.path.dirname(HERE), "include", "spec_kv.h"), os.path.join(CSRC, "fstream.cuh"),
                  os.path.join(os.path.dirname(HERE), "include", "spec_verify.h"),
                  os.path.join(os.path.dirname(HERE), "include", "spec_lm_head.h"),
                  os.path.join(os.path.dirname(HERE), "include", "spec_logprobs.h"),
                  os.path.join(os.path.dirname(HERE), "include", "spec_prompt.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in DEPS)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile libspec_verify.so next to this file; returns its path."""
    if not force and up_to_date():
        return LIB
    with tempfile.TemporaryDirectory() as tmp:
        # one compiler process per source, side by side, then the link
        jobs = []
        for src in SOURCES:
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            cmd = [nvcc(), *NVCC_FLAGS, *(extra or []), "-c", "-o", obj, src]
            if verbose:
                print(" ".join(cmd))
            jobs.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        done = [(p.communicate()[0], p.returncode) for _, p in jobs]
        link = [nvcc(), *NVCC_FLAGS, "-shared", "-o", LIB + ".tmp", *(obj for obj, _ in jobs)]
        if not any(rc for _, rc in done):
            if verbose:
                print(" ".join(link))
            res = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            done.append((res.stdout, res.returncode))
    for text, rc in done:
        if rc != 0:
            raise RuntimeError(f"nvcc failed ({rc}):\n{text}")
        if verbose and text:
            print(text)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose=True, extra=sys.argv[1:]))
