"""Build libmk.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m persistent_decode_megakernel_02_b200.build [--verbose]
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmk.so")
SOURCES = ["mk_kernel.cu", "mk_runtime.cpp", "mk_graph.cpp", "mk_static.cu", "mk_rows.cu",
           "mk_rows_graph.cpp", "mk_rows_runtime.cpp", "mk_ops.cpp", "mk_kv_append.cu",
           "mk_paged_attn.cu", "mk_prompt_attn.cu", "mk_sample.cu"]
HEADERS = ["mk_internal.h", "mk_ptx.cuh", "mk_rows.h", "mk_ops.h", "mk_ops.cuh", "mk_tc.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


STAMP = LIB + ".sha256"


def _digest() -> str:
    """Hash of every input of the build (sources, headers, flags)."""
    import hashlib
    h = hashlib.sha256()
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "mk.h"))
    for f in deps:
        h.update(os.path.basename(f).encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH).encode())
    return h.hexdigest()


def _stale() -> bool:
    # content-based: copies of the tree (which may not keep mtimes) reuse the
    # library as long as its inputs are unchanged
    if not os.path.exists(LIB) or not os.path.exists(STAMP):
        return True
    with open(STAMP) as f:
        return f.read().strip() != _digest()


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    cmd = [_nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-shared",
           "-I", os.path.join(ROOT, "include"), "-o", LIB]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += [os.path.join(CSRC, f) for f in SOURCES]
    subprocess.check_call(cmd)
    with open(STAMP, "w") as f:
        f.write(_digest())
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
