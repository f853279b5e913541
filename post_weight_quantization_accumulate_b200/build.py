"""Builds libgptq.so (sm_100a) in-tree from csrc/*.cu with nvcc, and the
CPython module _calls.so (the host side of w8a8.py) from csrc/calls.cpp with
the C++ compiler.

    python -m post_weight_quantization_accumulate_b200.build [--force] [--verbose]

Objects go to _build/ at the repository root; the libraries land next to this
file so they travel with the source tree.
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgptq.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
CALLS_STAMP = os.path.join(BUILD, "calls.txt")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "-I", os.path.join(ROOT, "include"), "-DNDEBUG"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "gptq.h")]


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def _calls_for() -> str:
    """What _calls.so is built for: another torch or Python needs another one."""
    import torch
    return f"torch {torch.__version__} python {sys.version}"


def calls_up_to_date() -> bool:
    if not _newer(CALLS, [CALLS_SRC, os.path.join(ROOT, "include", "gptq.h")]) or not os.path.exists(CALLS_STAMP):
        return False
    with open(CALLS_STAMP) as f:
        return f.read() == _calls_for()


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """_calls.so: torch's headers and libraries, and libgptq.so beside it."""
    if not force and calls_up_to_date():
        return CALLS
    import torch
    os.makedirs(BUILD, exist_ok=True)
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = CALLS + f".tmp{os.getpid()}"
    obj = os.path.join(BUILD, f"calls.{os.getpid()}.o")
    compile_ = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include"),
                "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(base, "include"),
                "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
                "-isystem", os.path.join(cuda, "include"), "-c", CALLS_SRC, "-o", obj]
    # linked by the C compiler, with the C++ runtime that torch has loaded instead of a copy of its
    # own: streams of a second, static one crashed where torch's had set up the locale
    link = [os.environ.get("CC", "gcc"), "-shared", obj, "-o", tmp, "-L", os.path.dirname(LIB), "-lgptq", "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-l:libstdc++.so.6", "-Wl,-rpath," + os.path.join(base, "lib")]
    try:
        for cmd in (compile_, link):
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"{cmd[0]} failed for {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, CALLS)
    finally:
        for left in (obj, tmp):
            if os.path.exists(left):
                os.remove(left)
    with open(CALLS_STAMP, "w") as f:
        f.write(_calls_for())
    return CALLS


def _calls_or_warning(force: bool, verbose: bool) -> None:
    """Only w8a8.py needs _calls.so: where it cannot be built, the library
    stands by itself, and w8a8 says what is missing when it is called."""
    try:
        build_calls(force, verbose)
    except Exception as e:   # no compiler, no headers, no torch
        if os.path.exists(CALLS):
            os.remove(CALLS)   # of older sources, or for another torch or Python
        warnings.warn(f"w8a8.py will not work: {e}", RuntimeWarning, stacklevel=3)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        _calls_or_warning(force, verbose)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = _sources()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if (verbose or ptxas_info) and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _calls_or_warning(force, verbose)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))
    sys.exit(0)
