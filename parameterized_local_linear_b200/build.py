"""Build libparallax.so in-tree with nvcc for sm_100a, and the tensor marshalling
module _marshal.so (csrc/marshal.cpp) that binding.py calls it through.

    python -m parameterized_local_linear_b200.build [--force] [--verbose]
"""
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libparallax.so")
SOURCES = [os.path.join(CSRC, f) for f in ("parallax_api.cu", "norm_rope_api.cu", "chunk_api.cu")]
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return [f for f in files if f.endswith((".cu", ".cuh", ".h"))]


def _newer(target, files) -> bool:
    return os.path.exists(target) and all(
        os.path.getmtime(f) <= os.path.getmtime(target) for f in files)


def up_to_date() -> bool:
    return _newer(LIB, _inputs()) and _newer(MARSHAL, [MARSHAL_SOURCE,
                                                       os.path.join(CSRC, "internal.h"),
                                                       os.path.join(INCLUDE, "parallax.h")])


def _build_marshal() -> None:
    import torch
    root = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    subprocess.run(
        ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-I", sysconfig.get_paths()["include"], "-I", inc,
         "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda, "-I", INCLUDE, "-I", CSRC,
         "-o", MARSHAL + ".tmp", MARSHAL_SOURCE, "-L", lib, "-lc10", "-lc10_cuda",
         "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-L", PKG, "-l:libparallax.so", "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(MARSHAL + ".tmp", MARSHAL)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
           "-std=c++17", "-t", "0", "-Xcompiler", "-fPIC", "-shared", "-I", INCLUDE, "-I", CSRC,
           "-Xlinker", "-soname,libparallax.so",
           "-o", LIB + ".tmp", *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    _build_marshal()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
