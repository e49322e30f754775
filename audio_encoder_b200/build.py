"""Builds libmoss_enc.so (all CUDA kernels + the C ABI) for sm_100a with nvcc,
and _pycalls.so (the Python side of the single-token calls) with g++.

Run from anywhere:  python -m audio_encoder_b200.build
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
MAIN = os.path.join(SRC_DIR, "moss_enc.cu")
LIB = os.path.join(HERE, "libmoss_enc.so")
HEADER = os.path.join(ROOT, "include", "moss_enc.h")
PYCALLS = os.path.join(SRC_DIR, "pycalls.cpp")
PYCALLS_LIB = os.path.join(HERE, "_pycalls.so")

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


def build_pycalls(force: bool = False) -> str:
    if not force and os.path.exists(PYCALLS_LIB) and \
            all(os.path.getmtime(s) <= os.path.getmtime(PYCALLS_LIB) for s in (PYCALLS, HEADER)):
        return PYCALLS_LIB
    import sysconfig
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = PYCALLS_LIB + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{t}/include",
           f"-I{t}/include/torch/csrc/api/include", f"-I{cuda}/include", f"-I{sysconfig.get_paths()['include']}",
           "-o", tmp, PYCALLS, f"-L{t}/lib", f"-Wl,-rpath,{t}/lib", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch", "-ltorch_python"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, PYCALLS_LIB)
    return PYCALLS_LIB


def build(force: bool = False, verbose: bool = False) -> str:
    build_pycalls(force)
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


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
