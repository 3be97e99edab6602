"""Build libfvattn.so (the CUDA path) in-tree with nvcc for sm_100a.

    python -m block_sparse_attention_aware_b200.build [--force]

Each .cu under csrc/ is compiled to an object with
`-gencode arch=compute_100a,code=sm_100a -lineinfo -O3` as a whole program
(no relocatable device code: ptxas honours per-warpgroup register budgets
only then), then linked into block_sparse_attention_aware_b200/libfvattn.so.
csrc/binding.cpp, a Python extension over that library's C ABI and torch's
tensors, becomes _native.so beside it, built again when torch or Python is
another than it was built for.  Needs nvcc, g++ and torch's headers (no GPU).
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfvattn.so")
NATIVE = os.path.join(HERE, "_native.so")
STAMP = os.path.join(BUILD, "native.txt")      # what _native.so was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

SOURCES = ["api.cu", "reorder.cu", "route.cu", "attn.cu", "noalloc.cu", "grad.cu", "cache.cu"]
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
         "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(f) for f in files)


def _fresh(path):
    return os.path.exists(path) and os.path.getmtime(path) >= _deps()


def native_target() -> str:
    """What _native.so is built for: it calls into this torch and this Python."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def _native_fresh():
    if not _fresh(NATIVE) or not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read() == native_target()


def _native_command():
    """g++ of binding.cpp against this interpreter's torch, to be linked with LIB."""
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    dirs = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DFV_NATIVE_TARGET="{native_target()}"',
            *(x for d in dirs for x in ("-isystem" if d != INCLUDE else "-I", d)), os.path.join(CSRC, "binding.cpp"),
            "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-L", HERE, "-l:libfvattn.so", "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not _fresh(LIB):
        _build_lib(verbose)
        force = True           # the extension is linked with it
    if force or not _native_fresh():
        os.makedirs(BUILD, exist_ok=True)
        tmp = NATIVE + f".tmp{os.getpid()}"
        subprocess.check_call([*_native_command(), "-o", tmp])
        os.replace(tmp, NATIVE)
        with open(STAMP, "w") as f:
            f.write(native_target())
    return LIB


def _build_lib(verbose: bool):
    os.makedirs(BUILD, exist_ok=True)
    objs, procs = [], []
    for src in SOURCES:   # the translation units compile in parallel
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [NVCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((cmd, subprocess.Popen(cmd)))
        objs.append(obj)
    for cmd, proc in procs:
        if proc.wait() != 0:
            raise subprocess.CalledProcessError(proc.returncode, cmd)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a",
                           "-o", tmp, *objs, "-lcudart"])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
