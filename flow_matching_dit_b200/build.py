"""In-tree build of the CUDA library ``libgdit.so`` for sm_100a.

``python -m flow_matching_dit_b200.build`` (or ``build()``) compiles
``csrc/gdit.cu`` (the action head) and ``csrc/ops.cu`` (the operators) with nvcc
into ``flow_matching_dit_b200/libgdit.so``, and ``csrc/binding.cpp`` (the
operators' Python calls) with the host compiler against torch's headers into
``_binding.so``.  With ``checked=True`` the library alone goes into ``libgdit_checked.so``, the range-checked build
(``-DGDIT_CHECKED=1``: guard bands around device allocations, index checks in
the kernels).  nvcc cross-compiles, so this works on a machine without a GPU.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libgdit.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = os.path.join(PKG, "csrc", "binding.cpp")
LIB_CHECKED = os.path.join(PKG, "libgdit_checked.so")
SOURCES = sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")) + glob.glob(os.path.join(PKG, "csrc", "*.cuh")))
HEADER = os.path.join(ROOT, "include", "gdit.h")


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdit.so")


def command(out: str = LIB, checked: bool = False) -> list:
    return [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
            "-Xcompiler", "-fPIC", "-shared", "-I" + os.path.join(ROOT, "include"),
            "-diag-suppress", "177"] + (["-DGDIT_CHECKED=1"] if checked else []) + \
        ["--threads", "2", "-o", out, os.path.join(PKG, "csrc", "gdit.cu"), os.path.join(PKG, "csrc", "ops.cu")]


def binding_command(out: str = BINDING) -> list:
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"), os.path.join(ROOT, "include"),
               sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + ["-I" + p for p in include] + \
        [BINDING_SOURCE, "-o", out, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
         "-lc10_cuda", "-lc10"]


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING):
        return False
    t = os.path.getmtime(BINDING)
    return all(os.path.getmtime(s) <= t for s in (BINDING_SOURCE, HEADER))


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(s) <= t for s in SOURCES + [HEADER])


def _run(cmd: list, tmp: str, out: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, out)


def binding_possible() -> bool:
    """Whether torch and Python's headers are here, which the binding needs and the library does not."""
    import importlib.util
    import sysconfig
    return importlib.util.find_spec("torch") is not None and \
        os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Builds what is not up to date; returns the library's path.  The operators' binding is built with the library, not
    with its checked form, and left out (and said so) where torch or Python's headers are missing: the operators' Python
    calls then raise, all else works."""
    out = LIB_CHECKED if checked else LIB
    if force or not up_to_date(out):
        tmp = out + ".tmp"
        _run(command(tmp, checked), tmp, out, verbose)
    if not checked and (force or not binding_up_to_date()):
        if binding_possible():
            tmp = BINDING + ".tmp"
            _run(binding_command(tmp), tmp, BINDING, verbose)
        else:
            print("torch or Python.h not found: the operators' Python calls are not built", file=sys.stderr)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, checked="--checked" in sys.argv))
