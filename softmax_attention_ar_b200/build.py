"""Build the ARL2 C-ABI library (libarl2.so) in-tree for sm_100a with nvcc.

    python -m softmax_attention_ar_b200.build [--force]

The library links the CUDA runtime statically and reaches the driver's tensor-map encoder
through cudaGetDriverEntryPoint, so it needs no libcuda at link time. ptxas resource
usage (registers, spills, shared memory) is written to _build/ptxas.log.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libarl2.so")
BUILD_DIR = os.path.join(PKG, "_build")
SOURCES = ["arl2_api.cu", "arl2_query.cu", "arl2_commit.cu", "arl2_clean.cu", "arl2_token.cu", "arl2_gates.cu",
           "arl2_noalloc.cu", "arl2_scan.cu", "arl2_attn.cu", "arl2_attn_fwd.cu", "arl2_attn_bwd.cu"]
HEADERS = ["arl2_device.cuh", "arl2_kernels.h", "arl2_query_body.cuh", "arl2_commit_rows.cuh", "arl2_attn.cuh",
           "arl2_attn_kernels.h"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the ARL2 library needs the CUDA 12.9 toolkit to build")


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "arl2.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-shared",
           "-Xptxas", "-v", "-I", os.path.join(ROOT, "include"),
           *[os.path.join(CSRC, f) for f in SOURCES], "-o", LIB + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(BUILD_DIR, "ptxas.log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stderr[-6000:]}")
    os.replace(LIB + ".tmp", LIB)
    if verbose:
        print(res.stderr)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
