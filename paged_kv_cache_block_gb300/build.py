"""Build libpagedkv.so in-tree: one nvcc process per translation unit (in parallel), then link.

    python -m paged_kv_cache_block_gb300.build [--force] [--ptxas-info]

Targets sm_103a only.  The CUDA runtime is linked statically; the driver API entry point the
library needs (TMA descriptor encoding) is looked up at run time, so building needs no GPU.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
SOURCES = ["api.cu", "slot_mapping.cu", "reshape_and_cache.cu", "paged_attention.cu", "noalloc.cu",
           "block_updates.cu", "block_manager.cpp", "prefill_attention.cu", "paged_decode_int4.cu",
           "selftest.cu", "paged_attention_fp8.cu", "build_batch.cu", "qk_norm_rope.cu", "tree_attention.cu",
           "tree_packed.cu", "paged_sinks.cu", "prefill_sinks.cu",
           "prefill_sinks_wide.cu"]
HEADERS = ["common.cuh", "dependent_launch.cuh", "tcgen05.cuh", "tree_common.cuh", "decode_common.cuh", "paged_decode_kernel.cuh", "prefill_sinks.cuh",
           "kernels.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, ptxas_info: bool = False, verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + sorted(glob.glob(os.path.join(ROOT, "include", "*.h")))
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str):
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
        if not (force or ptxas_info) and not _stale(o, [s] + hdrs):
            return o, ""
        cmd = [nvcc()] + ARCH + FLAGS + extra + ["-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return o, r.stderr

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    objs = [o for o, _ in results]
    if verbose or ptxas_info:
        for o, log in results:
            if log:
                sys.stderr.write(log)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, ptxas_info=args.ptxas_info, verbose=True))
