"""Builds the CUDA library ``libpmg.so`` in-tree with nvcc for sm_103a.

The translation units of ``csrc/`` are compiled in parallel, with one
``-gencode``, and linked with the CUDA runtime statically; no fast-math. The
library lands in ``paged_mla_kv_cache_gb300/lib/`` (git-ignored) and is rebuilt
when a source or a public header is newer than it.
"""
from __future__ import annotations

import os
import shutil
import subprocess

UNITS = ["mla_plan.cu", "mla_append.cu", "mla_decode.cu", "mla_decode_tc.cu", "mla_prefill.cu",
         "mla_prefill_tc.cu", "mla_bounds.cu", "mla_scores.cu", "mla_scores_tc.cu", "mla_select.cu", "mla_shared.cu",
         "mla_shared_tc.cu", "mla_shared_pair.cu", "mla_packed.cu"]
PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
SRC = os.path.join(CSRC, "pmg_gather.cu")
SOURCES = [SRC] + [os.path.join(CSRC, f) for f in UNITS]
HEADER = os.path.join(ROOT, "include", "pmg.h")
HEADERS = [HEADER, os.path.join(ROOT, "include", "pmg_mla.h"), os.path.join(ROOT, "include", "pmg_long.h")]
LIB_DIR = os.path.join(PKG_DIR, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libpmg.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
]
LINK_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-cudart", "static"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpmg.so")


def needs_build() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    shared = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    return any(os.path.getmtime(f) > t for f in (*SOURCES, *HEADERS, *shared, __file__))


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile libpmg.so if it is missing or stale; returns its path."""
    if not force and not needs_build():
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    objects = [f"{tmp}.{i}.o" for i in range(len(SOURCES))]
    common = [nvcc_path(), *NVCC_FLAGS, *(["-Xptxas=-v"] if verbose else []), "-I", os.path.join(ROOT, "include")]
    try:
        jobs = [(cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
                for cmd in ([*common, "-c", "-o", o, src] for o, src in zip(objects, SOURCES))]
        for cmd, out, rc in [(cmd, j.communicate()[0], j.returncode) for cmd, j in jobs]:
            if rc != 0:
                raise RuntimeError(f"nvcc failed ({rc}):\n{' '.join(cmd)}\n{out}")
            if verbose:
                print(out)
        cmd = [nvcc_path(), *LINK_FLAGS, "-o", tmp, *objects]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed ({res.returncode}):\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
