"""Build ``libkdaproj.so`` (sm_103a) in-tree with nvcc.

The translation units compile in parallel into ``_build/`` beside this file
and link into ``_build/libkdaproj.so`` (static CUDA runtime, no libcuda link:
the TMA descriptor encoder is fetched from the driver at run time).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libkdaproj.so")

SOURCES = [
    "kp_api.cu",
    "kp_cc.cu",
    "kp_cc_inst_lo_bf16.cu",
    "kp_cc_inst_hi_bf16.cu",
    "kp_cc_inst_lo_fp16.cu",
    "kp_cc_inst_hi_fp16.cu",
    "kp_cc_inst_proj.cu",
    "kp_cc_inst_ring_lo_bf16.cu",
    "kp_cc_inst_ring_hi_bf16.cu",
    "kp_cc_inst_ring_lo_fp16.cu",
    "kp_cc_inst_ring_hi_fp16.cu",
    "kp_tc05.cu",
    "kp_smallk.cu",
    "kp_noalloc.cu",
    "kp_mx4.cu",
    "kp_ffn_stream.cu",
    "kp_ffn_tile.cu",
    "kp_ffn_bwd.cu",
    "kp_ffn_api.cu",
]
HEADERS = ["kp_internal.cuh", "kp_cc_kernel.cuh", "kp_ffn.cuh", "kp_mx4.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3",
    "-lineinfo",
    "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-I", INCLUDE,
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_input() -> float:
    paths = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    paths.append(os.path.join(INCLUDE, "kdaproj.h"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link the library; returns its path. Skips work when the
    library is newer than every source."""
    os.makedirs(BUILD, exist_ok=True)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        return LIB
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
