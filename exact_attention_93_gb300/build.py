"""Builds libfattn.so in-tree with nvcc for sm_103a, and, where torch is installed,
the small native module through which its tensors reach part of the library (g++,
against that torch).  The library alone needs no torch.

Each CUDA translation unit is compiled in parallel, then linked into one
shared library next to this file.  The CUDA runtime is linked statically and
the driver API is reached through the runtime's entry-point query, so the
library loads on machines without a GPU driver (its symbols can be listed
there; nothing can run).
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfattn.so")
BIND = os.path.join(HERE, "_bind_torch.so")
BIND_STAMP = os.path.join(HERE, "_bind_torch.stamp")  # goes where the module goes
SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_noalloc.cu", "fa_serve_api.cu",
           "fa_rotary.cu", "fa_cache.cu", "fa_paged_few.cu", "fa_paged_many.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    """Whether libfattn.so is there and newer than its sources."""
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def have_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def torch_version() -> str:
    """The installed torch's own account of its build (version, CUDA, commit), read
    without importing it."""
    root = os.path.dirname(importlib.util.find_spec("torch").origin)
    with open(os.path.join(root, "version.py")) as f:
        return f"{root}\n{f.read()}"


def bind_stamp() -> str:
    """What the native module is bound to beside its sources."""
    return f"{sysconfig.get_config_var('SOABI')}\n{torch_version()}"


def bind_up_to_date() -> bool:
    """The same for the native module, and whether torch and Python are those it was
    built with."""
    try:
        with open(BIND_STAMP) as f:
            if f.read() != bind_stamp():
                return False
    except OSError:
        return False
    if not os.path.exists(BIND):
        return False
    t = os.path.getmtime(BIND)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compiles (if needed) the library and the native module, which is left out where
    there is no torch, and returns the path of libfattn.so."""
    want_lib = force or not up_to_date()
    want_bind = have_torch() and (force or not bind_up_to_date())
    if not want_lib and not want_bind:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(compile_bind) if want_bind else None
        if want_lib:
            link_library(list(ex.map(lambda src: compile_one(src, verbose, extra), SOURCES)))
        if want_bind:
            link_bind(*bind.result())
    return LIB


def compile_one(src, verbose, extra):
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def link_library(objs):
    tmp = LIB + f".tmp{os.getpid()}"
    run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], "link failed")
    os.replace(tmp, LIB)


def link_bind(obj, torch_lib):
    # the module finds libfattn.so beside itself, and torch's libraries in the
    # process that imports it
    tmp = BIND + f".tmp{os.getpid()}"
    run(["g++", "-shared", "-o", tmp, obj, "-L" + HERE, "-l:libfattn.so", "-L" + torch_lib,
         "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"],
        "link failed")
    os.replace(tmp, BIND)
    with open(BIND_STAMP, "w") as f:
        f.write(bind_stamp())


def run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")


def compile_bind():
    """The object file of bind_torch.cpp, and where torch's libraries are."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD, "bind_torch.o")
    run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I" + INCLUDE,
         "-I" + sysconfig.get_path("include"), "-isystem", os.path.join(root, "include"),
         "-isystem", os.path.join(cuda, "include"),
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-c", os.path.join(CSRC, "bind_torch.cpp"), "-o", obj], "g++ failed for bind_torch.cpp")
    return obj, os.path.join(root, "lib")


if __name__ == "__main__":
    verbose = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if verbose else []
    print(build(force=True, verbose=verbose, extra=extra))
