"""Build ``libqoq.so`` (the CUDA library) in-tree with nvcc for sm_100a, and
``_torch_calls.so`` (the calls from torch tensors into it) with g++.

    python -m w4a8_quantized_gemm_02_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libqoq.so")
CALLS = os.path.join(PKG, "_torch_calls.so")
CALLS_SRC = os.path.join(CSRC, "qoq_torch.cpp")
CALLS_STAMP = os.path.join(PKG, "_build", "_torch_calls.txt")   # what it was built against

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir() -> str:
    import importlib.util
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _built_against() -> str:
    """The installed torch (its version.py: version, commit, CUDA) and this Python: a module
    built against others has another binary interface."""
    torch = _torch_dir()
    with open(os.path.join(torch, "version.py")) as f:
        return f"{torch}\n{sys.version}\n{f.read()}"


def _calls_stale() -> bool:
    if not (os.path.exists(CALLS) and os.path.exists(CALLS_STAMP)):
        return True
    t = os.path.getmtime(CALLS)
    if any(os.path.getmtime(d) > t for d in (CALLS_SRC, os.path.join(INCLUDE, "qoq.h"))):
        return True
    with open(CALLS_STAMP) as f:
        return f.read() != _built_against()


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """The extension module, against the installed torch's headers."""
    import sysconfig
    if not force and not _calls_stale():
        return CALLS
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = CALLS + f".tmp{os.getpid()}"
    # torch's libraries are in the process already (torch is imported first); libqoq.so lies
    # beside the module
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
           "-I", os.path.join(torch, "include"), "-I", os.path.join(cuda, "include"),
           "-I", sysconfig.get_paths()["include"], CALLS_SRC, "-o", tmp,
           "-L", PKG, "-L", os.path.join(torch, "lib"), "-l:libqoq.so", "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.makedirs(os.path.dirname(CALLS_STAMP), exist_ok=True)
    if os.path.exists(CALLS_STAMP):
        os.remove(CALLS_STAMP)     # (no stamp of one build beside the module of another)
    os.replace(tmp, CALLS)
    with open(CALLS_STAMP, "w") as f:
        f.write(_built_against())
    return CALLS


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not _stale():
        build_calls(verbose=verbose)
        return LIB
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc(), *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
           "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    build_calls(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
