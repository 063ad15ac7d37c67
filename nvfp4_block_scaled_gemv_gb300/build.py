"""Build the in-tree shared library ``_lib/libnvfp4_gemv.so`` with nvcc (sm_103a).

Each CUDA translation unit is compiled in parallel, then linked with the
static CUDA runtime, so the library needs only the driver at run time.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")              # the GEMV and small-N GEMM kernels
CSRC_LAYER = os.path.join(HERE, "csrc_layer")  # the layer operators
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(OUT_DIR, "libnvfp4_gemv.so")
OBJ_DIR = os.path.join(HERE, "_build")

SOURCES = ["api.cu", "gemv_plain.cu", "gemv_permuted.cu", "gemv_async_plain.cu",
           "gemv_async_permuted.cu", "repack.cu", "gemv_tc.cu", "gemv_blockdot.cu",
           "gemv_blockwise.cu", "selftest.cu"]
LAYER_SOURCES = ["quantize.cu", "gemm_tc.cu", "gemm_pair.cu", "route.cu", "moe.cu", "layer_api.cu", "rope.cu",
                 "kv_cache.cu", "attention.cu", "attention_prompt.cu", "attention_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: set CUDA_HOME or put nvcc on PATH")
    return found


def _inputs() -> list[str]:
    files = [os.path.join(d, f) for d in (CSRC, CSRC_LAYER) for f in os.listdir(d)]
    files.append(os.path.join(INCLUDE, "nvfp4_gemv.h"))
    files.append(os.path.abspath(__file__))
    return files


def _up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library if any source is newer; returns its path."""
    if not force and _up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(OUT_DIR, exist_ok=True)

    def compile_one(src: str) -> str:
        folder = CSRC_LAYER if src in LAYER_SOURCES else CSRC
        obj = os.path.join(OBJ_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-I", CSRC_LAYER, "-c",
               os.path.join(folder, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
        if verbose:
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    sources = SOURCES + LAYER_SOURCES
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(sources)) as pool:
        objs = list(pool.map(compile_one, sources))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
