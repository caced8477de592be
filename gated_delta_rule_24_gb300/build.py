"""Build the sm_103a C-ABI library ``_build/libgdn_gb300.so`` in the package tree, and the
binding's extension ``_build/gdn_pycall.so`` beside it.

Each translation unit is compiled by nvcc in parallel, then linked; a rebuild
happens only when a source or header is newer than what is made of it.  The extension makes calls
lighter for the host and nothing else: where it cannot be built (no Python headers), the binding does
without.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig
import warnings

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


def _stale(made, deps) -> bool:
    return not os.path.exists(made) or any(os.path.getmtime(d) > os.path.getmtime(made) for d in deps)


def _build_pycall() -> None:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = PYCALL + f".tmp{os.getpid()}"
    try:
        r = subprocess.run(["gcc", "-O2", "-std=c11", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], "-I", INCLUDE,
                            "-I", os.path.join(cuda, "include"), PYCALL_SOURCE, "-o", tmp], capture_output=True, text=True)
        failed = r.returncode and f"gcc failed on {PYCALL_SOURCE}:\n{r.stdout}\n{r.stderr}"
    except OSError as e:
        failed = str(e)
    if not failed:
        os.replace(tmp, PYCALL)
        return
    if os.path.exists(PYCALL):  # of an older source
        os.remove(PYCALL)
    warnings.warn(f"calls of the decay operators will take the host longer: no {PYCALL}: {failed}")


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        extension = None
        if force or _stale(PYCALL, [PYCALL_SOURCE, os.path.join(INCLUDE, "gdn.h")]):
            extension = ex.submit(_build_pycall)
        if force or _stale(LIB, [os.path.join(CSRC, s) for s in SOURCES] + HEADERS):
            _build_lib(ex, verbose)
        if extension:
            extension.result()
    return LIB


def _build_lib(ex: cf.Executor, verbose: bool) -> None:
    nvcc = _nvcc()

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

    objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
