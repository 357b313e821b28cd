"""Build libattn_varlen.so in-tree with nvcc for sm_103a, and the native Python
entry points of the generation calls (_native.so) with the host compiler.

Each translation unit compiles in parallel; the objects are linked into one
shared library next to this file.  No GPU is needed to build.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libattn_varlen.so")
NATIVE = os.path.join(PKG, "_native.so")
OBJDIR = os.path.join(PKG, "_build")
SOURCES = ["host.cu", "sched.cu", "fwd.cu", "bwd_dq.cu", "bwd_dkdv.cu", "bwd_dkdv_drop.cu", "bwd_dkdv_dmask.cu",
           "noalloc.cu",
           "host_pipeline.cu", "shard.cu", "gate.cu",
           "cache_host.cu", "rotary.cu", "cache_fwd.cu", "cache_d160.cu", "cache_d128.cu",
           "cache_d64.cu", "cache_weights.cu", "evict.cu",
           "cache_more_host.cu", "norm.cu", "append8.cu", "cache8_fwd.cu", "cache8_d160.cu", "cache8_d128.cu",
           "cache8_d64.cu", "cache8_few_d160.cu", "cache8_few_d128.cu", "cache8_few_d64.cu", "pages.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xcompiler", "-Wall"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(os.path.dirname(PKG), "include", "attn_varlen.h"))
    return files


def build_native() -> None:
    """Compile _native.so against this interpreter's torch."""
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = NATIVE + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + sysconfig.get_paths()["include"], "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"),
           os.path.join(CSRC, "py_cache.cpp"), "-o", tmp, "-L" + libs, "-ltorch_python", "-ltorch_cpu",
           "-ltorch", "-lc10_cuda", "-lc10", "-Wl,-rpath," + libs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on py_cache.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, NATIVE)


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(NATIVE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(NATIVE))
    return any(os.path.getmtime(f) > t for f in _deps()) or os.path.getmtime(__file__) > t


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if stale) and return the path of libattn_varlen.so."""
    if not force and not _stale():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        return obj, res.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        native = ex.submit(build_native)
        results = list(ex.map(compile_one, SOURCES))
        native.result()
    if verbose or ptxas_info:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp] + [o for o, _ in results]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
