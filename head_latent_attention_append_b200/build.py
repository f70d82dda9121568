"""Builds libmla.so in-tree with nvcc for sm_100a (B200), and beside it the Python
module of the ragged-step calls (g++, torch's headers), which is linked to it."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmla.so")
MODULE = os.path.join(HERE, "_ragged.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-shared", "-Xptxas", "-v"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def up_to_date() -> bool:
    return _newer(LIB, sources() + [os.path.join(HERE, "..", "include", "mla.h")])


def _run(cmd, what: str, verbose: bool):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"building {what} failed")
    if verbose:
        sys.stderr.write(r.stderr)


def build_module(force: bool = False, verbose: bool = False) -> str:
    src = os.path.join(CSRC, "binding.cpp")
    if not force and _newer(MODULE, [src, os.path.join(HERE, "..", "include", "mla.h")]):
        return MODULE
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    includes = include_paths("cuda") + [sysconfig.get_paths()["include"]]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-isystem{d}" for d in includes), src,
          "-o", MODULE, "-L" + HERE, "-lmla", "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"], "_ragged.so", verbose)
    return MODULE


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not up_to_date():
        _run([NVCC, *FLAGS, "-o", LIB, os.path.join(CSRC, "mla_api.cu")], "libmla.so", verbose)
    build_module(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
