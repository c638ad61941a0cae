"""Builds libcarve.so (the C-ABI library of include/carve.h and carve_mixers.h) in-tree for sm_100a with nvcc, and
_carve_bind.so (the host side of the mixers' Python calls, against PyTorch's headers) with g++.  Without PyTorch
the library is built alone; with another PyTorch or Python than the last time the binding is built anew.

Each .cu file is compiled to an object in its own process (in parallel), then the objects are
linked into the shared library; an object is rebuilt only when its source, a header or this
file is newer than it."""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libcarve.so")
OBJ = os.path.join(PKG, "_build")
BIND = os.path.join(PKG, "_carve_bind.so")
BIND_FOR = os.path.join(PKG, "_carve_bind.for")   # what the built binding fits
BIND_SRC = os.path.join(PKG, "csrc", "carve_bind.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]


def sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cuh")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h"))) + [os.path.abspath(__file__)]


def deps():
    return sources() + headers()


def _obj(src):
    return os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in deps())


def bind_for() -> str | None:
    """What a binding fits, beside its sources: this PyTorch and this Python; None without PyTorch."""
    try:
        return f"torch {importlib.metadata.version('torch')} {sysconfig.get_config_var('EXT_SUFFIX')}"
    except importlib.metadata.PackageNotFoundError:
        return None


def bind_stale() -> bool:
    if bind_for() is None:   # nothing to build it against, or to call it from
        return False
    if not os.path.exists(BIND) or not os.path.exists(BIND_FOR):
        return True
    with open(BIND_FOR) as f:
        if f.read() != bind_for():
            return True
    t = os.path.getmtime(BIND)
    return any(os.path.getmtime(p) > t for p in [BIND_SRC, os.path.abspath(__file__)] +
               glob.glob(os.path.join(ROOT, "include", "*.h")))


def _bind(verbose):
    """Compiles and links the binding beside libcarve.so, which it finds in its own folder: by name, since by path
    (the library has no soname) a copied tree would load this one's."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    inc = os.path.join(torch, "include")
    cuda = os.path.dirname(os.path.dirname(os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")))
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w", "-I", inc, "-I",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"), "-I",
           sysconfig.get_paths()["include"], "-o", tmp, BIND_SRC, "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(torch, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BIND)
    with open(tmp, "w") as f:
        f.write(bind_for())
    os.replace(tmp, BIND_FOR)


def _compile(src, nvcc, force, verbose):
    obj = _obj(src)
    newest = max(os.path.getmtime(p) for p in [src] + headers())
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj
    tmp = obj + f".tmp{os.getpid()}"
    cmd = [nvcc, *FLAGS, *ARCH, "-I", os.path.join(ROOT, "include"), "-c", "-o", tmp, src]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, obj)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        if bind_stale():
            _bind(verbose)
        return LIB
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(lambda s: _compile(s, nvcc, force, verbose), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, "-shared", *ARCH, "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    if bind_stale() or (force and bind_for()):
        _bind(verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
