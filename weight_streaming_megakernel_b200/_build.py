"""Build libwsm.so in place with nvcc for sm_100a.

The library is plain CUDA C++ with a C ABI (include/wsm.h); this script is the
whole build.  ``python -m weight_streaming_megakernel_b200._build`` or
``build()`` from Python.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCES = ["wsm_api.cu", "wsm_umma.cu", "wsm_stream.cu", "wsm_noalloc.cu", "wsm_die.cu",
           "wsm_cache.cu", "wsm_experts.cu", "wsm_logprobs.cu", "wsm_opstatus.cu"]
HEADERS = ["wsm_internal.cuh", "wsm_tcgen05.cuh", "wsm_ops.cuh", "wsm_deal.cuh"]
LIB = os.path.join(PKG, "libwsm.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "wsm.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date(out: str = LIB) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=None, out: str = LIB) -> str:
    if not force and up_to_date(out):
        return out
    cmd = [nvcc(), *NVCC_FLAGS, *(extra_flags or []), "-I", os.path.join(ROOT, "include"), "-o", out,
           *[os.path.join(CSRC, f) for f in SOURCES]]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    tmp = out + ".tmp"
    cmd[cmd.index(out)] = tmp
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
