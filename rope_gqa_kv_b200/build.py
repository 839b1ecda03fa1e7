"""Build libgqa.so (all CUDA sources under csrc/) in-tree for sm_100a with nvcc.

    python -m rope_gqa_kv_b200.build [--force] [--verbose]

Each .cu is compiled to an object in _build/ (parallel), then linked into
rope_gqa_kv_b200/libgqa.so with the CUDA runtime linked statically.  A source
is rebuilt when it, or any header it may include, is newer than its object.
csrc/fastargs.c, the argument checks of the Python binding, becomes the extension
module rope_gqa_kv_b200/_fastargs.so (gcc), for one Python and one torch; where it does
not compile the binding checks in Python.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ_DIR = os.path.join(ROOT, "_build", "gqa")
LIB = os.path.join(PKG, "libgqa.so")
ARGS_SRC = os.path.join(CSRC, "fastargs.c")
ARGS_LIB = os.path.join(PKG, "_fastargs.so")
ARGS_FOR = os.path.join(OBJ_DIR, "fastargs.txt")          # what it was built for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgqa")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")))


def _compile(src: str, verbose: bool) -> tuple[str, str]:
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
    return obj, r.stderr


def _build_args(force: bool) -> None:
    import torch
    made_for = "python %s, torch %s\n" % (sys.version, torch.__version__)
    if not force and os.path.exists(ARGS_LIB) and os.path.exists(ARGS_FOR) and \
            open(ARGS_FOR).read() == made_for and os.path.getmtime(ARGS_LIB) >= max(
                os.path.getmtime(f) for f in [ARGS_SRC] + _headers()):
        return
    tmp = ARGS_LIB + ".tmp%d" % os.getpid()
    cmd = [shutil.which("gcc") or "gcc", "-O2", "-Wall", "-shared", "-fPIC",
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(os.path.dirname(torch.__file__), "include"), ARGS_SRC, "-o", tmp]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        err = r.stderr if r.returncode else None
    except OSError as e:
        err = str(e)
    if err is not None:                # the library works without it, but not with an old one
        if os.path.exists(ARGS_LIB):
            os.remove(ARGS_LIB)
        warnings.warn("gcc failed, arguments will be checked in Python:\n%s\n%s" %
                      (" ".join(cmd), err), RuntimeWarning)
        return
    os.replace(tmp, ARGS_LIB)
    with open(ARGS_FOR, "w") as f:
        f.write(made_for)


def build(force: bool = False, verbose: bool = False, jobs: int = 0) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    _build_args(force)
    srcs = _sources()
    newest_hdr = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    todo = []
    for s in srcs:
        obj = os.path.join(OBJ_DIR, os.path.basename(s) + ".o")
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(
                os.path.getmtime(s), newest_hdr):
            todo.append(s)
    logs = []
    if todo:
        with cf.ThreadPoolExecutor(max_workers=jobs or min(len(todo), os.cpu_count() or 4)) as ex:
            for obj, err in ex.map(lambda s: _compile(s, verbose), todo):
                logs.append(err)
    objs = [os.path.join(OBJ_DIR, os.path.basename(s) + ".o") for s in srcs]
    if todo or force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(
            os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
        os.replace(tmp, LIB)
    if verbose:
        sys.stderr.write("".join(logs))
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas resource usage")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
