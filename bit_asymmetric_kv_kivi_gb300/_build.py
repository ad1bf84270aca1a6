"""Builds the KIVI CUDA library (libkivi.so) in-tree with nvcc for sm_103a.

Each .cu translation unit is compiled in parallel, then linked into one
shared library with a plain C ABI (include/kivi.h). No torch headers are
involved, so the same library serves any PyTorch version.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libkivi.so")
OBJ_DIR = os.path.join(PKG, "_build")
SOURCES = ["kivi_abi.cu", "kivi_codec.cu", "kivi_decode.cu", "kivi_decode_k2v2.cu", "kivi_decode_k2v4.cu",
           "kivi_decode_k4v2.cu", "kivi_decode_k4v4.cu", "kivi_multi_k2v2.cu", "kivi_multi_k2v4.cu",
           "kivi_multi_k4v2.cu", "kivi_multi_k4v4.cu", "kivi_ext_k2v2.cu", "kivi_ext_k2v4.cu", "kivi_ext_k4v2.cu",
           "kivi_ext_k4v4.cu", "kivi_chunk_k2v2.cu", "kivi_chunk_k2v4.cu", "kivi_chunk_k4v2.cu", "kivi_chunk_k4v4.cu",
           "kivi_evict.cu", "kivi_noalloc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++20", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", f"-I{ROOT}/include"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the KIVI CUDA library cannot be built")
    return path


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "kivi.h")]
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libkivi.so (skipped when it is newer than every source)."""
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(OBJ_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
