"""Build libwmtp.so in-tree for sm_100a with nvcc, and the binding of its step
calls with the host compiler.

    python -m speculative_decode_draft_b200.build [--force]

Both are written next to this file so that they travel with the source
tree.  Rebuilds only what is older than one of its sources (or with --force).
libwmtp.so needs nvcc alone; where the binding, which needs a C++ compiler and
the headers of Python and PyTorch, cannot be built, only the step calls fail.
The binding's name has the versions of both, as it runs with no others.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

from . import _lib

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libwmtp.so")
SOURCES = [os.path.join(HERE, "csrc", "wmtp_abi.cu"), os.path.join(HERE, "csrc", "step_abi.cu"),
           os.path.join(HERE, "csrc", "page_pool.cpp"), os.path.join(HERE, "csrc", "selftest.cu")]
BINDING_SOURCE = os.path.join(HERE, "csrc", "step_binding.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libwmtp")


HEADERS = glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def _deps(out: str):
    if out != LIB:
        return [BINDING_SOURCE, *HEADERS]
    return [f for f in glob.glob(os.path.join(HERE, "csrc", "*")) if f != BINDING_SOURCE] + HEADERS


def up_to_date(out: str) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in _deps(out))


def _build_binding(out: str) -> None:
    """Against the headers and libraries of the PyTorch that imports it."""
    import torch
    home = os.path.dirname(torch.__file__)
    inc = os.path.join(home, "include")
    libs = os.path.join(home, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(ROOT, "include"), "-I" + sysconfig.get_paths()["include"], "-I" + inc,
           "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), "-I" + cuda, "-o", out + ".tmp",
           BINDING_SOURCE, "-L" + libs, "-Wl,-rpath," + libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the binding failed to build:\n" + r.stdout + r.stderr)
    os.replace(out + ".tmp", out)


def _build_library(verbose: bool) -> None:
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
           "-I" + os.path.join(ROOT, "include"), "-o", LIB + ".tmp", *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
    os.replace(LIB + ".tmp", LIB)
    if verbose:
        sys.stderr.write(r.stderr)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is out of date; the path of libwmtp.so.  A binding that cannot be built is a warning."""
    if force or not up_to_date(LIB):
        _build_library(verbose)
    try:
        binding = _lib.binding_path()
        if force or not up_to_date(binding):
            _build_binding(binding)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the step calls (wmtp_step.h) have no binding: {e}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    if not up_to_date(_lib.binding_path()):
        sys.exit(1)
