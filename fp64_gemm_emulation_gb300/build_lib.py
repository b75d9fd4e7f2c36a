"""Build libozaki.so (sm_103a) in-tree with nvcc: one object per .cu, compiled in parallel; and, beside it, the binding's
helper _tensor_lists.so (host code against torch's headers) with g++.

Usage: ``python -m fp64_gemm_emulation_gb300.build_lib`` (also called by
``__graft_entry__.build()``).  Objects go to ``fp64_gemm_emulation_gb300/_build/``,
the library to ``fp64_gemm_emulation_gb300/libozaki.so``; both are git-ignored.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libozaki.so")
LISTS = os.path.join(PKG, "_tensor_lists.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                     "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(obj: str, src: str, headers: list[str]) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(p) > t for p in [src] + headers)


def build_lists(verbose: bool = False, force: bool = False) -> str:
    """_tensor_lists.so, a Python module (csrc/tensor_lists.cpp).  It is bound to torch's and Python's binary interfaces: what it
    was built for stands beside the objects, and another torch or Python builds it anew."""
    import sysconfig

    import torch

    src, stamp = os.path.join(CSRC, "tensor_lists.cpp"), os.path.join(BUILD, "tensor_lists.for")
    built_for = f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, {sysconfig.get_config_var('SOABI')}"
    if not force and not _stale(LISTS, src, []) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == built_for:
                return ""
    root = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"], "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           src, "-o", LISTS + ".tmp", "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath," + lib]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(LISTS + ".tmp", LISTS)
    os.makedirs(BUILD, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(built_for)
    return r.stderr


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    todo = [(s, o) for s, o in zip(srcs, objs) if force or _stale(o, s, headers)]
    exe = nvcc()

    def compile_one(pair):
        src, obj = pair
        cmd = [exe] + NVCC_FLAGS + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(len(todo) + 1, os.cpu_count() or 1))) as ex:
        lists = ex.submit(build_lists, verbose, force)  # beside the objects; what it says comes after the library
        for msg in ex.map(compile_one, todo):
            if verbose and msg:
                print(msg, file=sys.stderr)
        if force or _stale(LIB, objs[0], objs):
            cmd = [exe] + ARCH + ["-shared", "-o", LIB + ".tmp"] + objs
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(LIB + ".tmp", LIB)
        try:
            lists.result()
        except Exception as e:  # the library is whole without it; the one call that wants it says so
            print(f"{os.path.basename(LISTS)} was not built (ozaki_clip_grad_norm of the binding needs it): {e}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv))
