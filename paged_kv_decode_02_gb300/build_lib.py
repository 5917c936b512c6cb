"""Build libpagedkv.so in-tree with nvcc for sm_103a (no CMake, no torch extension).

Each CUDA translation unit compiles in parallel; the objects link into
``paged_kv_decode_02_gb300/libpagedkv.so`` (cudart linked statically, the driver's
tensor-map encoder reached through the runtime's entry-point query, so no -lcuda).
Run ``python -m paged_kv_decode_02_gb300.build_lib`` or call :func:`build`.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")

SOURCES = ["api.cu", "append.cu", "merge.cu", "decode_bf16.cu", "decode_int8.cu",
           "decode_e4m3.cu", "decode_e5m2.cu", "noalloc.cu",
           "cascade.cu", "blocks.cu", "decode_tc.cu", "decode_tc_int8.cu", "decode_tc_e4m3.cu",
           "decode_tc_e5m2.cu", "rotate.cu", "gather.cu", "diff_bf16.cu", "diff_int8.cu",
           "diff_e4m3.cu", "diff_e5m2.cu", "diff_merge.cu", "decode_tree.cu", "decode_tree_int8.cu",
           "decode_tree_e4m3.cu", "decode_tree_e5m2.cu", "tree_bf16.cu", "tree_int8.cu",
           "tree_e4m3.cu", "tree_e5m2.cu", "tree_join.cu", "resize.cu", "keep.cu", "prompt.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _compile(nvcc, src, extra):
    obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
    cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
    return obj, r.stderr


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "pagedkv.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (if sources changed) and return the path of libpagedkv.so."""
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(lambda s: _compile(nvcc, s, list(extra_flags)), SOURCES))
    if verbose:
        for _, err in results:
            if err.strip():
                print(err, file=sys.stderr)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
