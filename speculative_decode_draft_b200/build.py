"""Build libwmtp.so in-tree for sm_100a with nvcc, and the binding of its step
calls (_step_binding.so) with the host compiler.

    python -m speculative_decode_draft_b200.build [--force]

Both are written next to this file so that they travel with the source
tree.  Rebuilds only when a source under csrc/ or include/ is newer than either
(or with --force).
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libwmtp.so")
SOURCES = [os.path.join(HERE, "csrc", "wmtp_abi.cu"), os.path.join(HERE, "csrc", "step_abi.cu"),
           os.path.join(HERE, "csrc", "page_pool.cpp"), os.path.join(HERE, "csrc", "selftest.cu")]
BINDING = os.path.join(HERE, "_step_binding.so")
BINDING_SOURCE = os.path.join(HERE, "csrc", "step_binding.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libwmtp")


def _deps():
    return (glob.glob(os.path.join(HERE, "csrc", "*")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
            + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(d) <= t for d in _deps())


def _build_binding() -> None:
    """Against the headers and libraries of the PyTorch that imports it."""
    import torch
    home = os.path.dirname(torch.__file__)
    inc = os.path.join(home, "include")
    libs = os.path.join(home, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(ROOT, "include"), "-I" + sysconfig.get_paths()["include"], "-I" + inc,
           "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), "-I" + cuda, "-o", BINDING + ".tmp",
           BINDING_SOURCE, "-L" + libs, "-Wl,-rpath," + libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the binding failed to build:\n" + r.stdout + r.stderr)
    os.replace(BINDING + ".tmp", BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    _build_binding()
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
           "-I" + os.path.join(ROOT, "include"), "-o", LIB + ".tmp", *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
    os.replace(LIB + ".tmp", LIB)
    os.utime(BINDING)  # both newer than their sources
    if verbose:
        sys.stderr.write(r.stderr)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
