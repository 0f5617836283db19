"""Build the KDA C-ABI shared library for sm_100a, and the binding of its paged operators.

    python -m gated_delta_rule_88_b200.build [--force]

Compiles every ``csrc/*.cu`` with nvcc (``-gencode arch=compute_100a,
code=sm_100a -O3 -lineinfo``) into ``_build/`` at the repository root and
links ``libkda_b200.so`` next to this file (in-tree, so it travels with the
repository to the GPU host).  ``csrc/binding.cpp`` is compiled by the host's
compiler against torch's headers into ``_paged.so`` beside it, after the library,
which needs nvcc alone.  Each is rebuilt only when a source or header of its own
is newer; the binding also when it was built for another torch or Python.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkda_b200.so")
BINDING = os.path.join(CSRC, "binding.cpp")
EXT = os.path.join(PKG, "_paged.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _built_for() -> str:
    """What a binding goes with, as it is written into the module."""
    import torch

    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def needs_binding() -> bool:
    if not os.path.exists(EXT):
        return True
    t = os.path.getmtime(EXT)
    if any(os.path.getmtime(p) > t for p in (BINDING, os.path.join(INCLUDE, "kda.h"))):
        return True
    with open(EXT, "rb") as f:
        return f"\0{_built_for()}\0".encode() not in f.read()


def build_binding(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_binding():
        return EXT
    import torch

    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    dirs = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = EXT + f".tmp{os.getpid()}"
    # (nvcc's own host compiler, whatever CXX says: a compiler without the shared C++ runtime links a second copy
    # of it into the module, whose streams then crash in a process that has torch's)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DKDA_BUILT_FOR="{_built_for()}"', *[x for d in dirs for x in ("-isystem", d)], BINDING, "-o", tmp, "-L", os.path.join(home, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {BINDING}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    return EXT


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    build_library(force, verbose, extra)
    build_binding(force, verbose)
    return LIB


def build_library(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and not needs_build():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    flags = FLAGS + (extra or [])

    def cc(pair):
        src, obj = pair
        cmd = [NVCC, *ARCH, *flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        for msg in ex.map(cc, zip(srcs, objs)):
            if verbose and msg:
                print(msg, flush=True)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    extra = [a for a in sys.argv[1:] if a.startswith("-X") or a.startswith("-D")]
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, extra=extra))
