"""Build the sm_103a CUDA library in-tree: nvcc compiles each translation unit (in parallel)
and links ``paged_kv_cache_134_gb300/lib/libpagedkv.so``.  No cmake, one -gencode."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libpagedkv.so")

SOURCES = ["api.cu", "append.cu", "decode.cu", "decode_f16.cu", "decode_bf16.cu", "decode_fp8_f16.cu",
           "decode_fp8_bf16.cu", "decode_tc.cu", "decode_mma.cu", "decode_mma_int4.cu",
           "decode_mma_int4_mass.cu", "decode_mma_fp8_mass.cu", "decode_mma_16bit_mass.cu",
           "decode_short.cu", "decode_short_fp8.cu", "decode_short_int4.cu", "evict.cu",
           "prefill.cu", "prefill_packed.cu", "prefill_paged.cu",
           "prefill_cascade.cu", "noalloc.cu", "blocks.cu", "selftest.cu",
           "prefix_cache.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    deps = _deps()
    extra = list(extra_flags or [])
    if os.environ.get("PAGEDKV_PTXAS_VERBOSE"):
        extra += ["-Xptxas", "-v"]
    objs = [os.path.join(BUILD, os.path.splitext(s)[0] + ".o") for s in SOURCES]
    todo = [(s, o) for s, o in zip(SOURCES, objs) if _stale(o, deps) or extra]

    def compile_one(so):
        src, obj = so
        cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return src, r.stderr

    if todo:
        with cf.ThreadPoolExecutor(max_workers=min(len(todo), os.cpu_count() or 4)) as ex:
            for src, err in ex.map(compile_one, todo):
                if verbose and err.strip():
                    print(f"--- {src}\n{err}", file=sys.stderr)
    if todo or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
