"""Builds libbonsai.so (the sm_100a CUDA library behind include/bonsai.h) in-tree.

    python -m ternary_weight_02_b200.build [--force] [--verbose-ptxas]

Each csrc/*.cu is compiled to an object under _build/ (in parallel, skipped when
up to date) and linked with the static CUDA runtime into
ternary_weight_02_b200/libbonsai.so.  csrc/pycall.c, the binding's fast call path, becomes
the extension module _bonsai_call.abi3.so beside it (gcc and the Python headers; Python's
stable ABI, so that one file serves every CPython from 3.10 on); where that cannot be built,
the binding makes the same calls through ctypes.  No GPU needed.
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

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libbonsai.so")
CALL_SRC = os.path.join(CSRC, "pycall.c")
CALL = os.path.join(PKG, "_bonsai_call.abi3.so")
HEADER = os.path.join(ROOT, "include", "bonsai.h")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libbonsai")
    return path


def _deps_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    files.append(HEADER)
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, force: bool, ptxas_verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if (not force and os.path.exists(obj)
            and os.path.getmtime(obj) >= max(os.path.getmtime(src), _deps_mtime())):
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
    if ptxas_verbose:
        print(res.stderr)
    return obj


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, force, ptxas_verbose), srcs))
    if (force or not os.path.exists(LIB)
            or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
    build_call(force)
    return LIB


def build_call(force: bool = False) -> str | None:
    """The extension module behind the per-layer entry points, or None (and a note) where there is
    no C compiler or no Python headers: the binding does without it."""
    old = os.path.join(PKG, "_bonsai_call.so")  # of builds for one interpreter; any other would load it too
    if os.path.exists(old):
        os.remove(old)
    if (not force and os.path.exists(CALL)
            and os.path.getmtime(CALL) >= max(os.path.getmtime(CALL_SRC), os.path.getmtime(HEADER))):
        return CALL
    tmp = CALL + ".tmp"
    cmd = [os.environ.get("CC", "gcc"), "-O2", "-shared", "-fPIC", "-DPy_LIMITED_API=0x030A0000", "-I",
           sysconfig.get_paths()["include"], CALL_SRC, "-o", tmp, "-L", PKG, "-l:libbonsai.so", "-Wl,-rpath,$ORIGIN"]
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
        note = res.stderr if res.returncode != 0 else None
    except OSError as e:
        note = str(e)
    if note is not None:
        print(f"{os.path.basename(CALL)} not built (calls go through ctypes): {note}", file=sys.stderr)
        if os.path.exists(CALL):
            os.remove(CALL)  # it belongs to older sources
        return None
    os.replace(tmp, CALL)
    return CALL


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.verbose_ptxas))
