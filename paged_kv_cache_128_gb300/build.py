"""Build libpagedkv.so in-tree: nvcc for the sm_103a kernels, g++ for the
host block manager, compiled in parallel and linked into one shared library
next to this file.  No torch extension machinery, no cmake."""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libpagedkv.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
HEADERS = [os.path.join(ROOT, "include", "pagedkv.h"), os.path.join(CSRC, "common.cuh"),
           os.path.join(CSRC, "tcgen05.cuh"), os.path.join(CSRC, "decode_tile.cuh"),
           os.path.join(CSRC, "decode_kernels.cuh"), os.path.join(CSRC, "prefill_common.cuh"),
           os.path.join(CSRC, "score_rules.cuh"), os.path.join(CSRC, "stage_ring.h"),
           os.path.join(CSRC, "token_rows.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]

CUDA_SOURCES = ["reshape_and_cache.cu", "paged_decode.cu", "paged_prefill.cu", "step_runner.cu",
                "rope_and_cache.cu", "shared_prefix.cu", "paged_decode_rules.cu",
                "paged_decode_rules_cap.cu", "paged_prefill_rules.cu"]
CXX_SOURCES = ["block_manager.cpp"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libpagedkv")


def _run(cmd):
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if proc.returncode != 0:
        raise RuntimeError("build step failed:\n" + " ".join(cmd) + "\n" + proc.stdout)
    return proc.stdout


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False, ptxas_info: bool = False) -> str:
    """Compile every translation unit and link ``libpagedkv.so``; return its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    jobs = []
    objs = []
    for src in CUDA_SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD_DIR, src + ".o")
        objs.append(obj)
        if force or _stale(obj, [path] + HEADERS):
            cmd = [nvcc, "-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
                   "-c", path, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)
    for src in CXX_SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD_DIR, src + ".o")
        objs.append(obj)
        if force or _stale(obj, [path] + HEADERS):
            cxx = os.environ.get("CXX", "g++")
            jobs.append([cxx, "-std=c++17", "-O2", "-fPIC", "-Wall", "-c", path, "-o", obj])
    if jobs:
        with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            outs = list(ex.map(_run, jobs))
        if verbose or ptxas_info:
            for cmd, out in zip(jobs, outs):
                print(" ".join(cmd))
                if out.strip():
                    print(out)
    if force or jobs or _stale(LIB_PATH, objs):
        _run([nvcc, "-shared", *ARCH, "-o", LIB_PATH, *objs, "-cudart", "static"])
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv, ptxas_info="--ptxas" in sys.argv))
