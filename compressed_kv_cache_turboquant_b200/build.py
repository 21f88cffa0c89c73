"""Compile the CUDA library ``libtq_b200.so`` in-tree for sm_100a.

    python compressed_kv_cache_turboquant_b200/build.py [-v] [-f]

(run it by path: importing the package loads the library it builds)

nvcc cross-compiles without a GPU.  The shared library exports the C ABI of
``include/tq.h`` and links the CUDA runtime statically, so loading it needs no
GPU (host-only entry points such as ``tq_make_codebook`` work anywhere).
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libtq_b200.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


# Kernels that move registers between their warpgroups (setmaxnreg): the
# assembler only does that in a unit compiled as a whole program.
WHOLE_PROGRAM = {"attn_tree.cu", "attn_tree_tc.cu", "attn_prompt.cu"}


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def build(verbose: bool = False, force: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        deps = [src] + [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))]
        deps.append(os.path.join(ROOT, "include", "tq.h"))
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(p) for p in deps):
            separate = src.endswith(".cu") and os.path.basename(src) not in WHOLE_PROGRAM
            cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-dc" if separate else "-c",
                   "-x", "cu" if src.endswith(".cu") else "c++", src, "-o", obj]
            if ptxas_verbose and src.endswith(".cu"):
                cmd[1:1] = ["-Xptxas", "-v"]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
        objs.append(obj)
    link = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", *objs, "-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(link), flush=True)
    subprocess.run(link, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv, ptxas_verbose="--ptxas" in sys.argv))
