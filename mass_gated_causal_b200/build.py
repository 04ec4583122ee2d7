"""Build the MALA CUDA library (sm_100a) in-tree: mass_gated_causal_b200/libmala.so,
and the torch side of some of its calls, mala_torch.so (csrc/mala_torch.cpp).

nvcc cross-compiles for sm_100a without a GPU. Every csrc/*.cu is one
translation unit, compiled to an object of its own (several at a time, and only
when one of the files it includes has changed, unless forced) and linked with
the static CUDA runtime, so the library carries no dependency on a particular
libcudart. It needs neither torch nor Python; the torch side is left out, with a
note, where torch is not installed. Run as a script (`python mass_gated_causal_b200/build.py`): the
package itself refuses to import while the library is missing.
"""
from __future__ import annotations

import importlib.util
import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
SRC_DIR = os.path.join(HERE, "csrc")
OBJ_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmala.so")
TORCH_SRC = os.path.join(SRC_DIR, "mala_torch.cpp")
TORCH_LIB = os.path.join(HERE, "mala_torch.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I" + os.path.join(os.path.dirname(HERE), "include")]


def sources():
    """The library's translation units."""
    return sorted(os.path.join(SRC_DIR, f) for f in os.listdir(SRC_DIR) if f.endswith(".cu"))


def _files_of(src):
    """A source and every file of this repository that it includes."""
    seen, todo = set(), [src]
    while todo:
        path = os.path.normpath(todo.pop())
        if path in seen:
            continue
        seen.add(path)
        with open(path) as f:
            todo += [os.path.join(os.path.dirname(path), x) for x in re.findall(r'^#include "([^"]+)"', f.read(), re.M)]
    return seen


def _object(src):
    return os.path.join(OBJ_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")


def _stale(out, files) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(f) > os.path.getmtime(out) for f in files)


def _has_torch() -> bool:
    """The C library needs no torch: without it only the torch side is left out."""
    return importlib.util.find_spec("torch") is not None


def needs_build() -> bool:
    return any(_stale(LIB, _files_of(s)) for s in sources()) or (_has_torch() and
                                                                 _stale(TORCH_LIB, _files_of(TORCH_SRC)))


def _build_torch_side() -> None:
    """mala_torch.so: a CPython module against torch's headers that calls libmala.so beside it."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    home = os.path.dirname(os.path.dirname(NVCC))
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += ["-isystem" + d for d in cpp_extension.include_paths() + [os.path.join(home, "include"),
                                                                     sysconfig.get_paths()["include"]]]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd += [TORCH_SRC, "-o", tmp, "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", LIB,
            "-Wl,-rpath,$ORIGIN"]
    subprocess.check_call(cmd)
    os.replace(tmp, TORCH_LIB)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)

    def compile_one(src):
        obj = _object(src)
        if force or _stale(obj, _files_of(src)):
            tmp = obj + f".tmp{os.getpid()}"
            subprocess.check_call([NVCC] + FLAGS + (["-Xptxas", "-v"] if verbose_ptxas else []) +
                                  ["-c", src, "-o", tmp])
            os.replace(tmp, obj)
        return obj

    with ThreadPoolExecutor(max_workers=min(len(sources()), os.cpu_count() or 1)) as pool:
        objs = list(pool.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC] + FLAGS + ["-shared", "-Xlinker", "-soname=libmala.so"] + objs + ["-o", tmp])
    os.replace(tmp, LIB)
    if not _has_torch():
        print("torch is not installed: mala_torch.so, the torch side of the calls beside attention, is not built")
    elif force or _stale(TORCH_LIB, _files_of(TORCH_SRC)):
        _build_torch_side()
    return LIB


if __name__ == "__main__":
    build(force="--changed" not in sys.argv, verbose_ptxas="-v" in sys.argv)
    print(LIB)
