"""Build libsffn.so (the HIP kernels and the C ABI) for gfx950, in-tree.

``python -m activation_sparse_feed_amd.build`` or ``build()`` from Python.
Each source is compiled to an object in parallel, then linked into
``activation_sparse_feed_amd/libsffn.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsffn.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.hip", "twell_gate.hip", "convert.hip", "dense.hip", "dense_skinny.hip", "sparse.hip",
           "route.hip", "norms.hip", "union.hip", "backward.hip", "backward_routed.hip", "probe.hip",
           "attn_api.hip", "heads.hip", "paged_attn.hip", "attn_rows_bf16.hip", "attn_rows_f32.hip",
           "attn_keys_bf16.hip", "attn_keys_f32.hip", "attn_mx4_api.hip", "heads_mx4.hip",
           "paged_attn_mx4.hip", "attn_mx4_rows_bf16.hip", "attn_mx4_rows_f32.hip",
           "attn_mx4_keys_bf16.hip", "attn_mx4_keys_f32.hip"]
ARCH = os.environ.get("SFFN_OFFLOAD_ARCH", "gfx950")

# Packed-FP32 instructions are kept out of the generated code.
HIPCC_FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Wno-unused-result", "-I", os.path.join(HERE, "..", "include")]


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP library cannot be built")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [_hipcc(), *HIPCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    """Compile every source and link libsffn.so; returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = min(len(SOURCES), max(1, min(16, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
