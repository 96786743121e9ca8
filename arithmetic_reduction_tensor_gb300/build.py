"""Compile libtcr (the CUDA kernels and the C ABI) for sm_103a, in-tree.

``python -m arithmetic_reduction_tensor_gb300.build`` or ``build_library()``
compiles every ``csrc/*.cu`` in parallel with nvcc and links
``_lib/libtcr.so`` (CUDA runtime linked statically, only the ``tcr_*``
symbols exported), and compiles ``csrc/bind.c``, the CPython module of the
8-bit path's calls, to ``_lib/_tcrbind.so`` with the host's C compiler.  Nothing is installed outside the source tree.
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libtcr.so")
BIND_SRC = os.path.join(CSRC, "bind.c")
BIND_PATH = os.path.join(OUT_DIR, "_tcrbind.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-Xptxas", "-warn-spills", "--ftz=false", "--prec-div=true", "--prec-sqrt=true",
              "--fmad=false", f"-I{INCLUDE}"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "tcr.h"))
    return sorted(hs)


def _stamp(extra: list[str]) -> str:
    h = hashlib.sha256()
    for p in _sources() + _headers() + [BIND_SRC]:
        with open(p, "rb") as f:
            h.update(p.encode() + b"\0" + f.read())
    h.update(" ".join(ARCH + NVCC_FLAGS + extra).encode())
    return h.hexdigest()


def _build_bind() -> None:
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    if not cc:
        raise RuntimeError("no C compiler: set CC or put gcc on PATH")
    tmp = f"{BIND_PATH}.{os.getpid()}.tmp"
    cmd = [cc, "-O2", "-Wall", "-shared", "-fPIC", f"-I{sysconfig.get_paths()['include']}", BIND_SRC, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cc} failed on {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND_PATH)


def build_library(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile and link ``_lib/libtcr.so``; skip when sources are unchanged."""
    extra = list(extra_flags or [])
    stamp = _stamp(extra)
    stamp_file = os.path.join(OUT_DIR, "libtcr.stamp")
    if (not force and os.path.exists(LIB_PATH) and os.path.exists(BIND_PATH)
            and os.path.exists(stamp_file)):
        with open(stamp_file) as f:
            if f.read().strip() == stamp:
                return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc = nvcc_path()

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    _build_bind()
    srcs = _sources()
    with ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = f"{LIB_PATH}.{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    with open(stamp_file, "w") as f:
        f.write(stamp + "\n")
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
