"""Build the in-tree shared library ``libgam.so`` (C ABI of include/gam.h).

Compiles every ``csrc/*.cu`` for sm_100a with nvcc (object files under
``_build/`` at the repository root, in parallel) and links them into
``conformer_speech_recognition_b200/libgam.so``.  nvcc cross-compiles, so this
runs on a machine without a GPU.  ``csrc/python_ops.cpp`` (the marshalling of
the streaming-block operators' Python calls) is compiled with g++ against torch's
headers into ``conformer_speech_recognition_b200/_ops.so`` beside it.  The library
itself needs nvcc alone: without torch the module is left out, and an error of its
compilation is raised after the library is there.

    python -m conformer_speech_recognition_b200.build [--force] [-j N]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgam.so")
OPS = os.path.join(PKG, "_ops.so")
OPS_MARK = "gam _ops built for "

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers_mtime() -> float:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(ROOT, "include", "gam.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, force: bool, hdr_mtime: float, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_mtime):
        return obj
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # a torch on the path that was not installed
        return "of unknown version"


def _built_for(path: str) -> bytes:
    """What a module was compiled against, from the mark that it holds (b"" if there is none)."""
    if not os.path.exists(path):
        return b""
    with open(path, "rb") as f:
        return f.read().partition(OPS_MARK.encode())[2].partition(b";")[0]


def _build_ops(force: bool) -> None:
    src = os.path.join(CSRC, "python_ops.cpp")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(ROOT, "include", "gam.h")))
    spec = importlib.util.find_spec("torch")
    if spec is None:
        print("torch is not installed: _ops.so, which its Python calls need, is not built", file=sys.stderr)
        return
    against = f"torch {_torch_version()} {sys.implementation.cache_tag}"
    if not force and os.path.exists(OPS) and os.path.getmtime(OPS) >= newest and _built_for(OPS) == against.encode():
        return
    torch = spec.submodule_search_locations[0]
    inc, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DGAM_BUILT_FOR="{OPS_MARK}{against};"', "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"), src, "-o", OPS + ".tmp",
           "-L", lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(OPS + ".tmp", OPS)


def build(force: bool = False, jobs: int = 8, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    hdr = _headers_mtime()
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        ops = ex.submit(_build_ops, force)
        objs = list(ex.map(lambda s: _compile(s, force, hdr, list(extra)), srcs))
    newest = max(os.path.getmtime(o) for o in objs)
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB, *objs, "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    ops.result()
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", type=int, default=8)
    ap.add_argument("--ptxas-v", action="store_true", help="print register / smem usage")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.ptxas_v else []
    try:
        build(force=a.force or a.ptxas_v, jobs=a.j, verbose=True, extra=extra)
    except RuntimeError as e:
        print(e, file=sys.stderr)
        sys.exit(1)
