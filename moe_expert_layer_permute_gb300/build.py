"""Builds the CUDA library `libmoe_gb300.so` in-tree for sm_103a with nvcc.

Each translation unit under `csrc/` is compiled in parallel, then linked into one shared library
with the CUDA runtime linked statically (the library needs no libcuda at load time: the driver
entry point for tensor-map encoding is looked up at run time).  Beside it `_marshal.so`, a Python
module that turns torch tensors into the library's arguments, from `csrc/marshal.cpp` with the host
compiler and torch's headers.  A stamp of the sources and flags skips the rebuild when nothing
changed.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libmoe_gb300.so")
MARSHAL = os.path.join(OUT_DIR, "_marshal.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the MoE layer library cannot be built")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _marshal_flags() -> list[str]:
    import torch
    top = os.path.dirname(torch.__file__)
    inc = os.path.join(top, "include")
    return ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I" + sysconfig.get_paths()["include"], "-I" + inc, "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
            "-I" + os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include"),
            "-L" + os.path.join(top, "lib"), f"-DTORCH_{torch.__version__.replace('.', '_').replace('+', '_')}"]


def _stamp(nvcc: str) -> str:
    h = hashlib.sha256()
    files = sources() + sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h", ".cpp")))
    files.append(os.path.join(ROOT, "include", "moe_layer.h"))
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join([nvcc] + ARCH + CFLAGS + _marshal_flags()).encode())
    h.update(os.uname().machine.encode())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of the shared library."""
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    stamp_file = os.path.join(OUT_DIR, "stamp")
    stamp = _stamp(nvcc)
    if not force and os.path.exists(LIB) and os.path.exists(MARSHAL) and os.path.exists(stamp_file):
        with open(stamp_file) as fh:
            if fh.read().strip() == stamp:
                return LIB

    def compile_one(src: str) -> str:
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *CFLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    flags = _marshal_flags()
    link = [f for f in flags if f.startswith("-L")]

    def compile_marshal() -> str:
        obj = os.path.join(OUT_DIR, "marshal.o")
        cmd = ["g++", *[f for f in flags if not f.startswith("-L")], "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on marshal.cpp:\n{r.stdout}\n{r.stderr}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(9, os.cpu_count() or 2)) as ex:
        marshal = ex.submit(compile_marshal)
        objs = list(ex.map(compile_one, sources()))
        marshal_obj = marshal.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = MARSHAL + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, marshal_obj, LIB, *link, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _marshal.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
