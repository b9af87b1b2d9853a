"""Build liblossk.so in-tree for sm_103a.

Each CUDA translation unit is compiled by its own nvcc process (in parallel),
then linked into ``output_projection_cross_gb300/_build/liblossk.so``.  The
CUDA runtime is linked statically, so the library needs only the driver.
Beside it stands ``_lossk_calls``, the CPython module through which the decoding
calls are made, named for the Python that it was built for.  Where that Python
has no headers it is left out: the losses need none of it, and the decoding
calls say so when one is made.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "liblossk.so")
CALLS = os.path.join(BUILD, "_lossk_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["lossk_abi.cu", "k_fwd2.cu", "k_bwp.cu", "k_simt.cu", "lossk_static.cu", "lossk_decode.cu", "k_beam.cu", "k_pages.cu",
           "k_attn.cu", "k_attn_mma.cu", "k_attn_ffma.cu", "lossk_seq.cu", "k_seq.cu", "k_rows.cu"]
HEADERS = ["ptx.cuh", "lossk_internal.h", "host_internal.h", "seq_internal.h", "seq_terms.cuh", "decode_internal.h", "decode_launch.h", "attn_split.cuh", "float2.cuh"]
CALLS_SOURCE = "lossk_calls.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build liblossk.so")


def _stale(path: str, sources: list) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    deps = [os.path.join(CSRC, f) for f in sources]
    deps.append(os.path.join(ROOT, "include", "lossk.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    python_h = sysconfig.get_paths()["include"]
    with cf.ThreadPoolExecutor(1) as ex:
        calls = None
        if not os.path.exists(os.path.join(python_h, "Python.h")):
            sys.stderr.write(f"no Python.h in {python_h}: the decoding calls' module is left out\n")
        elif force or _stale(CALLS, [CALLS_SOURCE]):
            calls = ex.submit(_build_calls, python_h)
        if force or _stale(LIB, SOURCES + HEADERS):
            _build_lib(verbose)
        if calls:
            calls.result()
    return LIB


def _build_calls(python_h: str) -> None:
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", python_h,
           os.path.join(CSRC, CALLS_SOURCE), "-o", tmp, "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed on {CALLS_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


def _build_lib(verbose: bool) -> None:
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if verbose:
        flags += ["-Xptxas", "-v"]
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
