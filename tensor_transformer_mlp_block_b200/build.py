"""Build step of the CUDA library: ``libtpmlp.so`` from ``csrc/tpmlp.cu``.

Compiled for sm_100a only (tcgen05 tensor cores, tensor memory and TMA are
Blackwell-datacenter features), in-tree, so the shared object sits beside the
binding that loads it.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtpmlp.so")
SOURCES = ["tpmlp.cu"]
HEADERS = ["ptx.cuh", "ckpt8.cuh", "gemm_tc.cuh", "gemm_tc2.cuh", "aux_kernels.cuh", "simt.cuh",
           "fused_kernels.cuh", "gemm_few.cuh", "norm.cuh", "fused_ops.cuh"]
INCLUDE = os.path.join(os.path.dirname(HERE), "include", "tpmlp.h")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-shared", "-Xcompiler", "-fPIC",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [INCLUDE]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, "-o", tmp, *[os.path.join(CSRC, s) for s in SOURCES]]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
