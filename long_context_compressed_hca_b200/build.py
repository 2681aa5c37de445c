"""Build libhca.so (the C-ABI library) and _torch_call.so in-tree.

Usage: python -m long_context_compressed_hca_b200.build [--force] [-v]
Each .cu under csrc/ is compiled by nvcc for sm_100a to an object in parallel,
then linked into long_context_compressed_hca_b200/libhca.so with the CUDA
runtime linked statically.  csrc/host/torch_call.cpp, the path from tensors to
some of its calls, becomes the extension module _torch_call.so, linked to
libhca.so and torch; libhca.so itself needs neither torch nor the extension, and
is linked before an error of the extension is raised.  Without torch there is no
extension.  Objects are rebuilt when their source or any header is newer.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libhca.so")
CALL_SRC = os.path.join(CSRC, "host", "torch_call.cpp")
CALL = os.path.join(PKG, "_torch_call.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(ROOT, "include", "hca.h"))
    return hs


def _compile(src: str, obj: str, extra, verbose: bool):
    cmd = [nvcc(), "-c", src, "-o", obj] + ARCH + FLAGS + list(extra)
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _run(cmd, what: str, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_call(obj: str, verbose: bool):
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    _run(["g++", "-c", CALL_SRC, "-o", obj, "-O2", "-std=c++17", "-fPIC", "-I" + os.path.join(ROOT, "include"),
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
          "-isystem", sysconfig.get_paths()["include"],
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"], "g++ torch_call.cpp", verbose)


def _link_call(obj: str, verbose: bool):
    import torch
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run(["g++", "-shared", "-o", CALL + ".tmp", obj, "-L" + tlib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
          "-lc10_cuda", "-L" + PKG, "-l:libhca.so", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + tlib], "link of _torch_call.so",
         verbose)
    os.replace(CALL + ".tmp", CALL)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))
    hdr_mtime = max(os.path.getmtime(h) for h in _headers())
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr_mtime):
            jobs.append((s, o))
    call_obj = os.path.join(BUILD, "torch_call.o")
    call_mtime = max(os.path.getmtime(CALL_SRC), os.path.getmtime(os.path.join(ROOT, "include", "hca.h")))
    has_torch = importlib.util.find_spec("torch") is not None
    call_job = has_torch and (force or not os.path.exists(call_obj) or os.path.getmtime(call_obj) < call_mtime)
    call = None
    if jobs or call_job:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs) + 1)) as ex:
            futs = {ex.submit(_compile, s, o, extra, verbose): s for s, o in jobs}
            if call_job:
                call = ex.submit(_compile_call, call_obj, verbose)
            for f in cf.as_completed(futs):
                warn = f.result()
                if verbose and warn.strip():
                    print(warn)
    if force or jobs or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        # a name of its own, so that _torch_call.so and a loader by path share one copy
        _run([nvcc(), "-shared", "-o", LIB + ".tmp"] + objs + ARCH +
             ["-cudart", "static", "-Xcompiler", "-fPIC", "-Xlinker", "-soname=libhca.so"], "link", verbose)
        os.replace(LIB + ".tmp", LIB)
    if call:
        call.result()
    if has_torch and (call_job or not os.path.exists(CALL) or os.path.getmtime(CALL) < os.path.getmtime(call_obj)):
        _link_call(call_obj, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
