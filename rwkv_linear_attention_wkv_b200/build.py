"""Builds libwkv.so (the CUDA library behind include/wkv.h) and _binding.so (the short way into
it from Python) in this package directory.

    python rwkv_linear_attention_wkv_b200/build.py [--verbose-ptxas] [--force]

(Run as a script, or load this file by path: importing it as a submodule would first
import the package, which needs the library this builds.)

nvcc compiles every csrc/*.cu for sm_100a only and links one shared library with the
CUDA runtime linked statically, so loading it needs no GPU and no torch. _binding.so is compiled
against the headers of the installed torch (found without importing it).
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libwkv.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """The library and, where torch is installed, the binding."""
    if force or verbose_ptxas or not up_to_date():
        build_library(verbose_ptxas)
    if importlib.util.find_spec("torch") is not None:
        build_binding(force)
    return LIB


def build_library(verbose_ptxas: bool = False) -> None:
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
           "-std=c++17", "-shared", "-Xcompiler", "-fPIC,-fvisibility=hidden",
           "--expt-relaxed-constexpr", "--threads", "0", "-I", INCLUDE, "-I", CSRC, "-o", LIB + ".tmp"]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    cmd += sources()
    subprocess.check_call(cmd)
    os.replace(LIB + ".tmp", LIB)


def torch_location() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def torch_version() -> str:
    with open(os.path.join(torch_location(), "version.py")) as f:
        return re.search(r"""__version__ = ['"](.+)['"]""", f.read()).group(1)


def binding_up_to_date() -> bool:
    """Newer than its sources, and built for the torch that is installed (it says so itself)."""
    if not os.path.exists(BINDING):
        return False
    t = os.path.getmtime(BINDING)
    if any(os.path.getmtime(p) > t for p in [BINDING_SOURCE] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return False
    with open(BINDING, "rb") as f:
        return f"built for torch {torch_version()}\0".encode() in f.read()


def build_binding(force: bool = False) -> str:
    """After build_library(): it links against the library."""
    if not force and binding_up_to_date():
        return BINDING
    torch = torch_location()
    cuda = os.path.dirname(os.path.dirname(NVCC))
    subprocess.check_call(
        [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
         f'-DTORCH_BUILT_FOR="{torch_version()}"', "-I", INCLUDE,
         "-I", os.path.join(torch, "include"), "-I", os.path.join(cuda, "include"),
         "-I", sysconfig.get_paths()["include"], BINDING_SOURCE, "-o", BINDING + ".tmp",
         "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
         "-L" + HERE, "-l:libwkv.so", "-Wl,-rpath,$ORIGIN"])
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="--verbose-ptxas" in sys.argv))
