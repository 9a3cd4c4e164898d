"""Builds libwq.so (the C-ABI library) from csrc/*.cu for sm_103a with nvcc, and _marshal.so
(Python argument marshalling, csrc/marshal.cpp, against the installed torch's headers).

Usage: ``python -m bit_weight_quantized_wq_gb300.build [--verbose-ptxas]``.
Objects go to ``_build/`` at the repository root; the library is written in-tree next to
this file.  Translation units compile in parallel.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libwq.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def build(verbose_ptxas: bool = False, quiet: bool = True) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                    "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, src[:-3] + ".o")
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        marshal = ex.submit(_compile_marshal)        # the slowest to compile: first
        results = list(ex.map(compile_one, srcs))
        marshal_obj = marshal.result()
    if verbose_ptxas or not quiet:
        for _, log in results:
            if log.strip():
                sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    _link_marshal(marshal_obj)
    return LIB


def _torch_flags():
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    flags = ["-O2", "-std=c++17", "-fPIC", "-w", "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)]
    return flags + [a for d in inc for a in ("-isystem", d)], os.path.join(root, "lib")


def _compile_marshal() -> str:
    obj = os.path.join(BUILD, "marshal.o")
    r = subprocess.run(["g++"] + _torch_flags()[0] + ["-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on marshal.cpp:\n%s\n%s" % (r.stdout, r.stderr))
    return obj


def _link_marshal(obj: str) -> None:
    tmp = MARSHAL + ".tmp"
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libwq.so", "-Wl,-rpath,$ORIGIN", "-L" + _torch_flags()[1],
                        "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of _marshal.so failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, MARSHAL)


if __name__ == "__main__":
    print(build(verbose_ptxas="--verbose-ptxas" in sys.argv, quiet=False))
