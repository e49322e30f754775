"""Builds libmoss_enc.so (all CUDA kernels + the C ABI) for sm_100a with nvcc,
and, where PyTorch is installed, the Python side of the single-token calls with
g++ against PyTorch's and Python's headers.

Run from anywhere:  python -m audio_encoder_b200.build [--force] [-v] [--lib]
(--lib: the library alone, for callers of the C ABI; it needs nvcc only)
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
MAIN = os.path.join(SRC_DIR, "moss_enc.cu")
LIB = os.path.join(HERE, "libmoss_enc.so")
HEADER = os.path.join(ROOT, "include", "moss_enc.h")
PYCALLS = os.path.join(SRC_DIR, "pycalls.cpp")

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared"]


def sources():
    return [os.path.join(SRC_DIR, f) for f in sorted(os.listdir(SRC_DIR))
            if f.endswith((".cu", ".cuh"))] + [HEADER]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


class PycallsError(RuntimeError):
    """The library is built, the Python side of the single-token calls is not."""


def pycalls_path() -> str:
    """Where the Python side of the single-token calls is built: it is bound to
    the interpreter's ABI and to PyTorch's, so its name has both."""
    import torch
    return os.path.join(HERE, f"_pycalls.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


def build_pycalls(force: bool = False) -> str:
    import torch
    lib = pycalls_path()
    if not force and os.path.exists(lib) and \
            all(os.path.getmtime(s) <= os.path.getmtime(lib) for s in (PYCALLS, HEADER)):
        return lib
    t = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{t}/include",
           f"-I{t}/include/torch/csrc/api/include", f"-I{cuda}/include", f"-I{sysconfig.get_paths()['include']}",
           "-o", tmp, PYCALLS, f"-L{t}/lib", f"-Wl,-rpath,{t}/lib", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch", "-ltorch_python"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    if not os.path.exists(nvcc) and os.path.exists("/usr/local/cuda/bin/nvcc"):
        nvcc = "/usr/local/cuda/bin/nvcc"
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, "-o", tmp, MAIN]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, and then the Python side of the single-token calls, whose
    failure is a PycallsError. Without PyTorch that side has no user and is left
    out."""
    build_library(force, verbose)
    if importlib.util.find_spec("torch") is None:
        print("PyTorch is not installed: the Python side of the single-token calls is not built", file=sys.stderr)
        return LIB
    try:
        build_pycalls(force)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        raise PycallsError(f"{LIB} is built, but not the Python side of the single-token calls: {e}") from e
    return LIB


if __name__ == "__main__":
    (build_library if "--lib" in sys.argv else build)(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
