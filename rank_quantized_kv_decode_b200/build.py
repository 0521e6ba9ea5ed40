"""Build ``libstarkv.so`` (sm_100a) in-tree with nvcc.

    python -m rank_quantized_kv_decode_b200.build [--verbose-ptxas]

The shared library lands next to this file, where the binding loads it from.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["api.cu", "decode.cu", "store.cu", "project.cu", "append_gemv.cu", "decode_noalloc.cu",
           "diag.cu", "absorb.cu", "hybrid.cu", "kv_api.cu", "kv_append.cu", "kv_select.cu", "kv_decode.cu"]
LIB = os.path.join(HERE, "libstarkv.so")


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    deps = srcs + [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith(".cuh")]
    deps.append(os.path.join(HERE, "..", "include", "starkv.h"))
    if not force and os.path.exists(LIB):
        lib_t = os.path.getmtime(LIB)
        if all(os.path.getmtime(d) <= lib_t for d in deps):
            return LIB
    flags = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
             "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]
    if verbose_ptxas:
        flags = ["-Xptxas", "-v"] + flags

    def run(args: list[str]) -> str:
        proc = subprocess.run([nvcc_path(), *args], cwd=CSRC, capture_output=True, text=True)
        if proc.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + proc.stdout + proc.stderr)
        return proc.stdout + proc.stderr

    # the sources side by side, then one link
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(os.cpu_count()) as pool:
        objs = [os.path.join(tmp, os.path.basename(s) + ".o") for s in srcs]
        logs = list(pool.map(lambda so: run([*flags, "-c", "-o", so[1], so[0]]), zip(srcs, objs)))
        run([*flags, "-shared", "-o", LIB + ".tmp", *objs])
    if verbose_ptxas:
        sys.stderr.write("".join(logs))
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose_ptxas="--verbose-ptxas" in sys.argv, force=True))
