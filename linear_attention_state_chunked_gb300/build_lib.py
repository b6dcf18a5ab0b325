"""Builds liblinstate.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each translation unit compiles in parallel; the link uses the static CUDA
runtime, so the library loads on machines without a GPU driver (the driver
entry points it needs are looked up at run time).
"""

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
LIB = os.path.join(PKG, "liblinstate.so")

# prompt_api.cu holds step_api.cu and that api.cu, whose checks and error text they share
SOURCES = ["prompt_api.cu", "copy_kernels.cu", "token_kernels.cu", "chunked_prefill.cu", "verify_chunk.cu",
           "selftest.cu", "kv_cache.cu", "attn_decode.cu", "attn_d64.cu", "attn_d128.cu",
           "attn_d256.cu", "attn_umma_d64.cu", "attn_umma_d128.cu", "attn_umma_d256.cu", "block_norm.cu",
           "kv_plan.cu", "rope.cu", "chunk_attn.cu", "chunk_mma_d64.cu", "chunk_mma_d128.cu", "chunk_mma_d256.cu",
           "chunk_umma_d64.cu", "chunk_umma_d128.cu", "chunk_umma_d256.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _deps():
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hdrs += [os.path.join(ROOT, "include", f) for f in ("lin_state.h", "lin_step.h", "lin_prompt.h")]
    hdrs += [os.path.join(CSRC, f) for f in ("api.cu", "step_api.cu")]
    return hdrs


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = _deps()
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or not _newer(o, [s] + hdrs):
            jobs.append([nvcc(), *ARCH, *FLAGS, *extra_flags, "-c", s, "-o", o])
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        for cmd, res in zip(jobs, ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs)):
            if verbose or res.returncode:
                sys.stderr.write(res.stdout + res.stderr)
            if res.returncode:
                raise RuntimeError("nvcc failed: " + " ".join(cmd))
    if force or jobs or not _newer(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("link failed: " + " ".join(cmd))
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
