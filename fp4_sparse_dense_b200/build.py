"""Builds the SharQ CUDA library (libsharq.so) in-tree with nvcc for sm_100a.

Usage: python -m fp4_sparse_dense_b200.build [--force]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIB_DIR, "libsharq.so")
SOURCES = ["sharq_api.cu", "prep.cu", "quant_weight.cu", "gemm.cu", "gemm_pair.cu",
           "noalloc.cu", "matvec.cu", "matvec_tile.cu", "tokens.cu"]
HEADERS = ["fp4_device.cuh", "fp4_quant.cuh", "sm100_ptx.cuh", "sharq_internal.h",
           "epilogue.cuh", "experts_internal.h", "matvec_device.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_input() -> float:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "sharq.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _run(cmd: list[str]) -> subprocess.CompletedProcess:
    return subprocess.run(cmd, capture_output=True, text=True)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(LIB_DIR, exist_ok=True)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        return LIB
    tmp = LIB + ".tmp"
    base = [nvcc(), *NVCC_FLAGS, *(extra_flags or []), "-I", os.path.join(ROOT, "include")]
    # the sources do not depend on one another: one nvcc each, a link at the end
    with tempfile.TemporaryDirectory(dir=LIB_DIR) as objects, ThreadPoolExecutor(os.cpu_count() or 1) as pool:
        objs = [os.path.join(objects, f[:-3] + ".o") for f in SOURCES]
        cmds = [[*base, "-c", "-o", o, os.path.join(CSRC, f)] for f, o in zip(SOURCES, objs)]
        link = [*base, "-shared", "-cudart", "static", "-o", tmp, *objs]
        for cmd, r in [*zip(cmds, pool.map(_run, cmds)), (link, _run(link))]:
            if verbose:
                print(" ".join(cmd))
                if r.stdout or r.stderr:
                    print(r.stdout, r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
