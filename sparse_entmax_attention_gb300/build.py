"""Build libentmaxkv.so in-tree for sm_103a (nvcc, one process per source).

``python -m sparse_entmax_attention_gb300.build`` or ``build_library()``.
Objects go to ``_build/`` beside this file, the shared library next to it.
Rebuilds only what is older than its sources.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libentmaxkv.so")

SOURCES = ["api.cu", "append.cu", "score.cu", "select.cu", "decode.cu", "softmax.cu", "noalloc.cu",
           "moment_fit.cu", "q8_api.cu", "pages.cu", "q8_append.cu", "q8_attend.cu", "q8_chunk.cu",
           "q8_chunk_i8_d128.cu", "q8_chunk_i8_d64.cu", "q8_chunk_e4m3_d128.cu", "q8_chunk_e4m3_d64.cu",
           "q8_entmax.cu", "q8_weigh.cu", "q8_evict.cu", "q8_weigh_chunk.cu",
           "q8_weigh_chunk_i8_d128.cu", "q8_weigh_chunk_i8_d64.cu", "q8_weigh_chunk_e4m3_d128.cu",
           "q8_weigh_chunk_e4m3_d64.cu", "q8_chunk_diff_i8_d128.cu", "q8_chunk_diff_i8_d64.cu",
           "q8_chunk_diff_e4m3_d128.cu", "q8_chunk_diff_e4m3_d64.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libentmaxkv")


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hs + [os.path.join(INCLUDE, "entmaxkv.h")]


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_library(verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    hdrs = _headers()
    extra = list(extra_flags or [])
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if _stale(o, [s] + hdrs):
            jobs.append([cc, *ARCH, *FLAGS, *extra, "-c", s, "-o", o])
    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        for cmd, res in zip(jobs, ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs)):
            if res.returncode != 0:
                raise RuntimeError("nvcc failed: %s\n%s%s" % (" ".join(cmd), res.stdout, res.stderr))
            if verbose and (res.stdout or res.stderr):
                print(res.stdout + res.stderr)
    if _stale(LIB, objs):
        cmd = [cc, *ARCH, "-shared", "-o", LIB, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed: %s\n%s%s" % (" ".join(cmd), res.stdout, res.stderr))
    return LIB


if __name__ == "__main__":
    print(build_library(verbose="-v" in sys.argv))
