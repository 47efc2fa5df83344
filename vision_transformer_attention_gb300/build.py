"""Builds libvta_gb300.so, the CUDA library behind include/rpe_attn.h, and
vta_bind.so, an extension module that makes small calls of it quickly.

Each .cu file under csrc/ is compiled for sm_103a only (one -gencode, so the
library runs on GB300 and nowhere else) in parallel, then linked into one
shared library in ``_build/``. Run ``python -m vision_transformer_attention_gb300.build``
or ``__graft_entry__.build()``.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libvta_gb300.so")
BIND = os.path.join(BUILD, "vta_bind.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr


def _bind_object():
    """bind.cpp's object, against the headers of the torch that is installed."""
    import torch
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "bind.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", base, "-isystem", os.path.join(base, "torch", "csrc", "api", "include"),
           "-isystem", cuda]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{res.stdout}\n{res.stderr}")
    return obj


def _bind_link(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, LIB, "-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of vta_bind.so failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BIND)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "rpe_attn.h"))
    bind_src = os.path.join(CSRC, "bind.cpp")
    newest = max(os.path.getmtime(p) for p in srcs + headers + [bind_src])
    if not force and all(os.path.exists(f) and os.path.getmtime(f) >= newest for f in (LIB, BIND)):
        return LIB
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(16, len(srcs) + 1)) as ex:
        bind = ex.submit(_bind_object)
        results = list(ex.map(lambda s: _compile(s, verbose), srcs))
        bind_obj = bind.result()
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-Xlinker", "-soname=libvta_gb300.so", "-o", tmp, *[o for o, _ in results], "-lcudart"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    _bind_link(bind_obj)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
