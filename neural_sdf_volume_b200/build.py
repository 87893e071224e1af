"""Builds libvdm.so (all CUDA sources under csrc/) for sm_100a, and _seq.so (the Python
calls of the token-sequence operators, against torch's headers), in-tree.

Usage: ``python -m neural_sdf_volume_b200.build`` or ``build()`` from Python.
Objects go to ``_build/`` next to this file; the shared libraries are
``libvdm.so`` and ``_seq.so`` in this package directory.  Without torch (and a C++ compiler
for its headers) the C library is built all the same; ``_seq.so`` is rebuilt when torch or Python change.
"""
from __future__ import annotations

import glob
import importlib.metadata
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libvdm.so")
SEQ = os.path.join(PKG, "_seq.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _deps_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*")) + [os.path.join(ROOT, "include", "vdm.h"), __file__]
    return max(os.path.getmtime(f) for f in files)


def _binding_versions() -> str | None:
    """What _seq.so is built against, beside the sources; None without torch."""
    try:
        return f"torch {importlib.metadata.version('torch')}, python {sys.version}"
    except importlib.metadata.PackageNotFoundError:
        return None


def _binding_fresh() -> bool:
    versions, stamp = _binding_versions(), os.path.join(BUILD, "seq_binding.versions")
    if versions is None:
        return True
    if not (os.path.exists(SEQ) and os.path.exists(stamp)) or os.path.getmtime(SEQ) < _deps_mtime():
        return False
    with open(stamp) as f:
        return f.read() == versions


def _compile_binding() -> str:
    """The object of csrc/seq_binding.cpp (it needs the Python and torch of this interpreter)."""
    from torch import _C
    from torch.utils.cpp_extension import include_paths
    obj = os.path.join(BUILD, "seq_binding.cpp.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(_C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda]
    for p in include_paths():
        cmd += ["-isystem", p]
    _run([*cmd, "-c", os.path.join(CSRC, "seq_binding.cpp"), "-o", obj], "compiling seq_binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    from torch.utils.cpp_extension import library_paths
    tmp = SEQ + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN"]
    for p in library_paths():
        cmd += ["-L", p]
    _run([*cmd, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], "linking _seq.so")
    os.replace(tmp, SEQ)
    with open(os.path.join(BUILD, "seq_binding.versions"), "w") as f:
        f.write(_binding_versions())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"{what} failed")


def build(force: bool = False, verbose: bool = False, extra: list | None = None) -> str:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime() and _binding_fresh():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = extra or []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError(f"nvcc failed for {src}")
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        binding = ex.submit(_compile_binding) if _binding_versions() else None
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    _run([NVCC, *ARCH, "-shared", "-Xlinker", "-soname=libvdm.so", "-o", tmp, *objs], "linking libvdm.so")
    os.replace(tmp, LIB)
    if binding is None:
        sys.stderr.write("torch not found: _seq.so (the Python calls of the token-sequence operators) not built\n")
    else:   # the C library stands whatever comes of this
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
