"""Build libmk.so (the C-ABI library) in-tree with nvcc for sm_100a, and the
binding's compiled fast path (_mk_fast.so) with g++ against torch's headers.

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


def _stale(lib: str = LIB, digest=None) -> bool:
    # content-based: copies of the tree (which may not keep mtimes) reuse the
    # library as long as its inputs are unchanged
    stamp = lib + ".sha256"
    if not os.path.exists(lib) or not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        return f.read().strip() != (digest or _digest)()


# Kernels that move registers between their warps: the shares add up to those of
# a launch with exactly this many a thread (kLaunchRegs, kLaunchRegsPrompt), and
# the library refuses to launch them with any other number.
LAUNCH_REGISTERS = {"mk_step_kernel": 168, "prompt_attn_kernel": 168}


def check_registers(log: str):
    """Raise if `log`, what nvcc -Xptxas -v printed, shows another number of
    registers for one of LAUNCH_REGISTERS, or none: the build would give a
    library that refuses that kernel's calls."""
    import re
    seen = set()
    for entry, n in re.findall(r"Compiling entry function '(\w+)'(?:(?!Compiling entry).)*?Used (\d+) registers", log, re.S):
        for name, want in LAUNCH_REGISTERS.items():
            if name in entry:
                seen.add(name)
                if int(n) != want:
                    raise RuntimeError(f"{entry} was compiled to {n} registers a thread; its split needs {want}")
    if missing := sorted(set(LAUNCH_REGISTERS) - seen):
        raise RuntimeError(f"the compiler named no registers for {', '.join(missing)}")


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _stale():
        cmd = [_nvcc(), "-O3", "-std=c++17", *ARCH, "-t", "0", "-lineinfo", "-Xcompiler", "-fPIC", "-shared",
               "-I", os.path.join(ROOT, "include"), "-o", LIB, "-Xptxas", "-v"]
        cmd += [os.path.join(CSRC, f) for f in SOURCES]
        done = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        if verbose or done.returncode:
            sys.stderr.write(done.stdout)
        if done.returncode:
            raise subprocess.CalledProcessError(done.returncode, cmd)
        try:
            check_registers(done.stdout)
        except RuntimeError:
            os.remove(LIB)
            raise
        with open(STAMP, "w") as f:
            f.write(_digest())
    build_fast(force)
    return LIB


FAST = os.path.join(HERE, "_mk_fast.so")
FAST_SOURCE = os.path.join(CSRC, "mk_fast.cpp")


def _fast_digest() -> str:
    """Hash of the fast path's source, the header and the versions it binds to."""
    import hashlib
    import torch
    h = hashlib.sha256(f"{torch.__version__} {sys.version}".encode())
    for f in (FAST_SOURCE, os.path.join(ROOT, "include", "mk.h")):
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def build_fast(force: bool = False) -> str:
    if not force and not _stale(FAST, _fast_digest):
        return FAST
    import sysconfig
    import torch
    base = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.isabs(_nvcc()) else "/usr/local/cuda"
    subprocess.check_call(
        ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-isystem", os.path.join(base, "include"),
         "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
         "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
         "-I", os.path.join(ROOT, "include"), "-o", FAST, FAST_SOURCE, "-L", HERE, "-lmk",
         "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"])
    with open(FAST + ".sha256", "w") as f:
        f.write(_fast_digest())
    return FAST


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
