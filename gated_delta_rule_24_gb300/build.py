"""Build the sm_103a C-ABI library ``_build/libgdn_gb300.so`` in the package tree, and the
binding's extension ``_build/gdn_pycall.so`` beside it.

Each translation unit is compiled by nvcc in parallel, then linked; a rebuild
happens only when a source or header is newer than the library or the extension.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgdn_gb300.so")
PYCALL = os.path.join(BUILD, "gdn_pycall.so")
PYCALL_SOURCE = os.path.join(CSRC, "pycall.c")
SOURCES = ["prefill.cu", "decode.cu", "decay_prefill.cu", "decay_step.cu", "norm_rope.cu", "api.cpp"]
HEADERS = [os.path.join(CSRC, f) for f in ("prefill.h", "decode.h", "decay.h", "decay.cuh", "ptx.cuh")] + [os.path.join(INCLUDE, "gdn.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(PYCALL):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(PYCALL))
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS + [PYCALL_SOURCE]
    return any(os.path.getmtime(d) > t for d in deps)


def _build_pycall() -> None:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = PYCALL + f".tmp{os.getpid()}"
    r = subprocess.run(["gcc", "-O2", "-std=c11", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], "-I", INCLUDE,
                        "-I", os.path.join(cuda, "include"), PYCALL_SOURCE, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on {PYCALL_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, PYCALL)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        extension = ex.submit(_build_pycall)
        objs = list(ex.map(compile_one, SOURCES))
        extension.result()
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
