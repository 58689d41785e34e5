"""Builds the CUDA library `libmoe_gb300.so` in-tree for sm_103a with nvcc.

Each translation unit under `csrc/` is compiled in parallel, then linked into one shared library
with the CUDA runtime linked statically (the library needs no libcuda at load time: the driver
entry point for tensor-map encoding is looked up at run time).  Beside it `_marshal.so`, a Python
module that turns torch tensors into the library's arguments for the balance loss and the
orthogonalisation, from `csrc/marshal.cpp` with the host compiler and Python's and torch's headers; where
those are missing the library is built all the same, with a warning, and only those calls cannot be made.
A stamp of the sources and flags skips each rebuild when nothing changed.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sysconfig
import warnings

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


def _stamp(files: list[str], flags: list[str]) -> str:
    h = hashlib.sha256()
    for f in files + [os.path.join(ROOT, "include", "moe_layer.h")]:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(flags).encode())
    h.update(os.uname().machine.encode())
    return h.hexdigest()


def _current(product: str, stamp_file: str, stamp: str) -> bool:
    if not (os.path.exists(product) and os.path.exists(stamp_file)):
        return False
    with open(stamp_file) as fh:
        return fh.read().strip() == stamp


def _run(cmd: list[str], what: str) -> subprocess.CompletedProcess:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def _build_marshal(force: bool) -> str:
    """The object of marshal.cpp, or "" where `_marshal.so` is current."""
    flags = _marshal_flags()
    source = os.path.join(CSRC, "marshal.cpp")
    if not force and _current(MARSHAL, MARSHAL + ".stamp", _stamp([source], flags)):
        return ""
    obj = os.path.join(OUT_DIR, "marshal.o")
    _run(["g++", *[f for f in flags if not f.startswith("-L")], "-c", source, "-o", obj], "g++ on marshal.cpp")
    return obj


def _link_marshal(obj: str) -> None:
    flags = _marshal_flags()
    tmp = MARSHAL + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, LIB, *[f for f in flags if f.startswith("-L")], "-ltorch_python", "-ltorch_cpu", "-ltorch",
          "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"], "link of _marshal.so")
    os.replace(tmp, MARSHAL)
    with open(MARSHAL + ".stamp", "w") as fh:
        fh.write(_stamp([os.path.join(CSRC, "marshal.cpp")], flags))


def _build_library(nvcc: str, force: bool, verbose: bool) -> None:
    stamp_file = os.path.join(OUT_DIR, "stamp")
    headers = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h")))
    stamp = _stamp(sources() + headers, [nvcc] + ARCH + CFLAGS)
    if not force and _current(LIB, stamp_file, stamp):
        return

    def compile_one(src: str) -> str:
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        r = _run([nvcc, *ARCH, *CFLAGS, "-c", src, "-o", obj], f"nvcc on {src}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of the shared library."""
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        marshal = ex.submit(_build_marshal, force)
        _build_library(nvcc, force, verbose)
        try:
            if obj := marshal.result():
                _link_marshal(obj)
        except (RuntimeError, OSError, ImportError) as e:
            warnings.warn(f"the balance loss and the orthogonalisation cannot be called, marshalling was not built: {e}")
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
