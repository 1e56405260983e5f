"""Builds libkda.so in-tree for sm_103a with nvcc (one -gencode, objects compiled in
parallel, no cmake).  ``python -m gated_delta_rule_55_gb300.build_lib`` or ``build()``."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libkda.so")
SOURCES = ["kda_abi.cu", "kda_decode.cu", "kda_chunk_simt.cu", "kda_chunk_tc.cu",
           "kda_chunk_split.cu", "kda_noalloc.cu", "kda_recurrent.cu", "kda_backward.cu",
           "kda_gla.cu", "kda_gla_chunk.cu", "kda_chunk_bwd.cu", "kda_selftest.cu", "kda_step.cu",
           "kda_norm_rope.cu", "kda_cache_q8.cu", "kda_paged_attn.cu", "kda_paged_attn_q8.cu",
           "kda_paged_q8_few.cu", "kda_paged_q8_few32.cu", "kda_paged_attn_prefix.cu",
           "kda_paged_attn_prefix_q8.cu", "kda_paged_attn_simt.cu", "kda_serving_abi.cu"]
HEADERS = ["kda_internal.cuh", "tc_prims.cuh", "chunk_common.cuh", "chunk_records.cuh",
           "kda_paged.cuh", "kda_paged_line.h", "kda_paged_tc.cuh", "kda_paged_plan.cuh",
           "kda_paged_q8_few.cuh", "kda_q8.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"),
]


def _nvcc():
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libkda")
    return p


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every CUDA source of the library and link libkda.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "kda.h")]
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        list(ex.map(run, jobs))
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    if force or jobs or _stale(LIB_PATH, objs):
        run([nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", *objs,
             "-o", LIB_PATH])
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
