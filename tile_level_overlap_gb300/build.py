"""Build libmk.so in-tree with nvcc for sm_103a (no cmake, parallel objects)."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmk.so")

SOURCES = ["mk_plan.cpp", "mk_capi.cu", "mk_k_generic.cu", "mk_k_h1_f4_d64_r4.cu",
           "mk_k_h2_f7_d128_r4.cu", "mk_k_h2_f6_d128_r4.cu", "mk_gemm.cu", "mk_noalloc.cu",
           "mk_prefill_plan.cpp", "mk_prefill_kernel.cu", "mk_bdecode_plan.cpp",
           "mk_bdecode_kernel.cu", "mk_paged.cu", "mk_paged_few.cu", "mk_paged_chunk.cu"]
HEADERS = ["mk_internal.h", "mk_plan.h", "mk_device.cuh", "mk_kernel.cuh", "mk_variants.h",
           "mk_tc.cuh", "mk_tmap.h", "mk_prefill.h", "mk_bdecode.h", "mk_paged.h", "mk_paged_dev.cuh", "mk_paged_tc.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "mk.h")]
    common = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"] + ARCH
    jobs = []
    objs = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src + ".o")
        objs.append(obj)
        if _stale(obj, [path] + hdrs):
            cmd = [nvcc(), "-c", path, "-o", obj] + common + list(extra_flags)
            if src.endswith(".cu"):
                cmd += ["-Xptxas", "-v"] if verbose else []
            else:
                cmd = [nvcc(), "-x", "c++", "-c", path, "-o", obj] + common + list(extra_flags)
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=max(1, len(jobs))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError("nvcc failed: " + " ".join(cmd))
    if jobs or _stale(LIB, objs):
        cmd = [nvcc(), "-shared", "-o", LIB] + objs + ARCH + ["-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
