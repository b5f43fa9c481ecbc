"""Build libparallax.so in-tree with nvcc for sm_100a, and, where torch is
installed, the tensor marshalling module _marshal.so (csrc/marshal.cpp) that
binding.py calls it through. The library itself needs no torch.

    python -m parameterized_local_linear_b200.build [--force] [--verbose]
"""
import importlib.util
import os
import re
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


def torch_version():
    """The installed torch's version, without importing it; None if there is none."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    with open(os.path.join(spec.submodule_search_locations[0], "version.py")) as f:
        return re.search(r"^__version__ = '(.*)'", f.read(), re.M).group(1)


def _lib_up_to_date() -> bool:
    return _newer(LIB, _inputs())


def _marshal_up_to_date(torch_ver) -> bool:
    """Newer than its sources and built against this torch (marshal.cpp keeps the
    version as a string: the module follows torch's C++ ABI)."""
    if not _newer(MARSHAL, [MARSHAL_SOURCE, os.path.join(CSRC, "internal.h"),
                            os.path.join(INCLUDE, "parallax.h")]):
        return False
    with open(MARSHAL, "rb") as f:
        return f"built for torch {torch_ver}\0".encode() in f.read()


def up_to_date() -> bool:
    ver = torch_version()
    return _lib_up_to_date() and (ver is None or _marshal_up_to_date(ver))


def _build_lib(verbose: bool) -> None:
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
           "-std=c++17", "-t", "0", "-Xcompiler", "-fPIC", "-shared", "-I", INCLUDE, "-I", CSRC,
           "-Xlinker", "-soname,libparallax.so",
           "-o", LIB + ".tmp", *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)


def _build_marshal(torch_ver) -> None:
    import torch
    root = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    subprocess.run(
        ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         f'-DPLX_TORCH_VERSION="{torch_ver}"',
         "-I", sysconfig.get_paths()["include"], "-I", inc,
         "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda, "-I", INCLUDE,
         "-I", CSRC, "-o", MARSHAL + ".tmp", MARSHAL_SOURCE, "-L", lib, "-lc10", "-lc10_cuda",
         "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-L", PKG, "-l:libparallax.so",
         "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(MARSHAL + ".tmp", MARSHAL)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not _lib_up_to_date():
        _build_lib(verbose)
    ver = torch_version()
    if ver is not None and (force or not _marshal_up_to_date(ver)):
        _build_marshal(ver)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
