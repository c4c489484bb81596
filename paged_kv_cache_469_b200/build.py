"""Build libpa.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc, and the
Python module ``_binding`` (argument marshalling) with g++.  The library needs nvcc
alone; where torch is not installed the module, which is of no use there, is left out.

    python -m paged_kv_cache_469_b200.build [--force]

Objects go to ``paged_kv_cache_469_b200/_build/``; the shared library to
``paged_kv_cache_469_b200/libpa.so``, the module beside it.  Sources are
recompiled when they (or the headers) are newer than their object.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpa.so")
BINDING = os.path.join(PKG, "_binding.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, force: bool, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if (not force and os.path.exists(obj)
            and os.path.getmtime(obj) >= max(os.path.getmtime(src), _headers_mtime())):
        return obj
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas:
        sys.stderr.write(res.stderr)
    return obj


def _binding(force: bool) -> str | None:
    """The Python module, against the installed torch's headers and libraries (None
    without torch)."""
    import sysconfig

    try:
        import torch
    except ImportError as e:
        print(f"_binding left out: {e}", file=sys.stderr)
        return None
    src = os.path.join(CSRC, "binding.cpp")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "pa.h")))
    # an exchanged torch or Python is no newer file: what the module was built for
    # stands beside the objects
    mark = os.path.join(BUILD, "binding.built_for")
    now = f"{torch.__version__} {torch.__file__} {sys.version}"
    if (not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest
            and os.path.exists(mark)):
        with open(mark) as f:
            if f.read() == now:
                return BINDING
    root = os.path.dirname(torch.__file__)
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", "/usr/local/cuda/include",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", src, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
           "-ldl"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING)
    with open(mark, "w") as f:
        f.write(now)
    return BINDING


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        module = ex.submit(_binding, force)
        objs = list(ex.map(lambda s: _compile(s, force, verbose_ptxas), srcs))
        _link(objs, force)  # whatever becomes of the module
        module.result()
    return LIB


def _link(objs: list[str], force: bool) -> None:
    if (force or not os.path.exists(LIB)
            or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
