"""Build the SAW-INT4 CUDA library in-tree: bit_paged_kv_gb300/_build/libsaw_int4.so.

Each translation unit is compiled for sm_103a only (one -gencode), in
parallel, then linked into one shared library exporting the C ABI of
include/saw_int4.h.  Beside it goes _saw_step, a small CPython extension
through which Python makes the serving step's calls, under the interpreter's
own suffix; where the interpreter has no headers it is left out, and only
those calls are missing.  No torch headers are involved.
"""
from __future__ import annotations

import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libsaw_int4.so")
STEP = os.path.join(OUT_DIR, "_saw_step" + importlib.machinery.EXTENSION_SUFFIXES[0])

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
# (source, object, extra flags).  The append kernel's bytes are defined by
# separately rounded binary32 steps; it uses explicit _rn intrinsics and is
# also compiled with contraction off.  The decode kernel is built once per CTA
# shape (16, 8 and 4 warps), once more with 16 and 8 warps for head_dim 64
# and 256, once more per shape as the shared-prefix decode's second pass, and
# per shape and size for lists of pages; the rotary append again with norms.
UNITS = [("saw_api.cu", "saw_api.o", []),
         ("quantize_append.cu", "quantize_append.o", ["-fmad=false"]),
         ("paged_decode.cu", "paged_decode_w16.o", ["-DSAW_DECODE_WARPS=16"]),
         ("paged_decode.cu", "paged_decode_w8.o", ["-DSAW_DECODE_WARPS=8"]),
         ("paged_decode.cu", "paged_decode_w4.o", ["-DSAW_DECODE_WARPS=4"]),
         ("paged_decode.cu", "paged_decode_dims_w16.o",
          ["-DSAW_DECODE_WARPS=16", "-DSAW_DECODE_OTHER_DIMS"]),
         ("paged_decode.cu", "paged_decode_dims_w8.o",
          ["-DSAW_DECODE_WARPS=8", "-DSAW_DECODE_OTHER_DIMS"]),
         ("paged_decode.cu", "paged_decode_shared_w16.o",
          ["-DSAW_DECODE_WARPS=16", "-DSAW_DECODE_SHARED"]),
         ("paged_decode.cu", "paged_decode_shared_w8.o",
          ["-DSAW_DECODE_WARPS=8", "-DSAW_DECODE_SHARED"]),
         ("paged_decode.cu", "paged_decode_shared_w4.o",
          ["-DSAW_DECODE_WARPS=4", "-DSAW_DECODE_SHARED"]),
         ("paged_decode.cu", "paged_decode_sparse_w16.o",
          ["-DSAW_DECODE_WARPS=16", "-DSAW_DECODE_SPARSE"]),
         ("paged_decode.cu", "paged_decode_sparse_w8.o",
          ["-DSAW_DECODE_WARPS=8", "-DSAW_DECODE_SPARSE"]),
         ("paged_decode.cu", "paged_decode_sparse_w4.o",
          ["-DSAW_DECODE_WARPS=4", "-DSAW_DECODE_SPARSE"]),
         ("paged_decode.cu", "paged_decode_sparse_dims_w16.o",
          ["-DSAW_DECODE_WARPS=16", "-DSAW_DECODE_OTHER_DIMS", "-DSAW_DECODE_SPARSE"]),
         ("paged_decode.cu", "paged_decode_sparse_dims_w8.o",
          ["-DSAW_DECODE_WARPS=8", "-DSAW_DECODE_OTHER_DIMS", "-DSAW_DECODE_SPARSE"]),
         ("prefix_attn.cu", "prefix_attn.o", []),
         ("build_tables.cu", "build_tables.o", []),
         ("rope_append.cu", "rope_append.o", []),
         ("rope_append.cu", "rope_append_norm.o", ["-DSAW_ROPE_NORM"]),
         ("page_summary.cu", "page_summary.o", []),
         ("select_pages.cu", "select_pages.o", []),
         ("paged_decode_bf16.cu", "paged_decode_bf16.o", []),
         ("prefill_attn.cu", "prefill_attn.o", []),
         ("variants.cu", "variants.o", []),
         ("decode_static_scratch.cu", "decode_static_scratch.o", [])]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "saw_int4.h"))
    files.append(os.path.abspath(__file__))
    return files


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    newest = max(os.path.getmtime(f) for f in _deps())

    def fresh(path: str) -> bool:
        return not force and os.path.exists(path) and os.path.getmtime(path) >= newest

    with ThreadPoolExecutor(max_workers=1) as ex:
        step = None if fresh(STEP) else ex.submit(_build_step)
        if not fresh(LIB):
            _build_lib(verbose)
        if step is not None:
            step.result()  # (the library is there whatever became of the extension)
    return LIB


def _build_step() -> None:
    headers = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(headers, "Python.h")) or not shutil.which("g++"):
        if os.path.exists(STEP):
            os.remove(STEP)  # of older sources
        sys.stderr.write(f"_saw_step is not built: no Python.h in {headers}, or no g++; the serving step's calls are "
                         "missing from Python\n")
        return
    tmp = STEP + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I", INCLUDE, "-I", headers,
           os.path.join(CSRC, "step_binding.cpp"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for step_binding.cpp:\n{r.stderr}")
    os.replace(tmp, STEP)


def _build_lib(verbose: bool) -> None:
    nvcc = _nvcc()

    def compile_one(unit) -> str:
        src, obj_name, extra = unit
        obj = os.path.join(OUT_DIR, obj_name)
        cmd = [nvcc, *ARCH, *COMMON, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(UNITS)) as ex:
        objs = list(ex.map(compile_one, UNITS))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
