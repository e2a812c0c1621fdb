"""Build libikbo.so (the sm_103a kernels + C ABI) in-tree with nvcc.

    python -m broadcast_gemm_attention_gb300.build [--force]

Each .cu file is compiled in parallel (one -gencode: compute_103a/sm_103a),
then linked into ``broadcast_gemm_attention_gb300/libikbo.so`` with the
static CUDA runtime.  ptxas register/spill reports go to
``broadcast_gemm_attention_gb300/_build/ptxas.log``.
"""
from __future__ import annotations

import argparse
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
LIB = os.path.join(PKG, "libikbo.so")
SOURCES = ["seg.cu", "lce.cu", "lce_noalloc.cu", "lce_bwd.cu", "attn.cu", "attn_bwd.cu", "rope.cu",
           "qcache.cu", "qattn.cu", "qattn_tile.cu", "qtree.cu", "linattn.cu", "linback.cu", "lintile.cu", "linread.cu", "api.cu",
           "qcache_api.cu", "linattn_api.cu"]
HEADERS = ["ptx.cuh", "ikbo_internal.h", "bwd_internal.h", "plan_internal.h", "qcache_internal.h",
           "attn_common.cuh", "mma_common.cuh", "tile_common.cuh", "linattn_internal.h", "launch.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "ikbo.h"), __file__]
    return max(os.path.getmtime(p) for p in paths)


def _compile(src: str) -> tuple:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
           "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return src, obj, r.returncode, r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(_compile, SOURCES))
    log = []
    for src, obj, rc, out in results:
        log.append(f"==== {src}\n{out}")
        if rc != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{out}")
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write("\n".join(log))
    if verbose:
        print("\n".join(log))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp] + [r[1] for r in results] + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
    sys.exit(0)
