"""Build libpgf8.so (the CUDA kernels + C ABI) in-tree for sm_100a.

Usage: python precision_gemm_fp8_b200/build.py [--force] [--verbose-ptxas]
(run it by path: importing the package loads the library this script builds)
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libpgf8.so")
SOURCES = ["pgf8_api.cu"]
DEPS = ["pgf8_api.cu", "gemm.cuh", "gemm_persistent.cuh", "gemm_streamk.cuh", "gemm_2sm.cuh", "gemm_group.cuh", "quantize.cuh", "sm100_ptx.cuh",
        "kvcache.cuh", "attention.cuh", "attention_context.cuh", "gemm_pair_group.cuh", "gemm_persistent_swap.cuh",
        "block_api.cuh", "gemm_block.cuh", "quantize_blocks.cuh", "packed_ptx.cuh",
        "moe_api.cuh", "moe.cuh", "gemm_block_pair.cuh"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpgf8")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, d) for d in DEPS] + [os.path.join(INCLUDE, "pgf8.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
           "-shared", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC, "-o", tmp] + [os.path.join(CSRC, s) for s in SOURCES]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libpgf8.so")
    if ptxas_verbose or not quiet:
        sys.stderr.write(res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.verbose_ptxas, quiet=False))
