"""Build step of libsbn.so: nvcc for sm_100a, in-tree, no JIT cache.

    python -m sparse_linear_layers_fwd_b200.build [--verbose]
"""

from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsbn.so")
SOURCES = [os.path.join(CSRC, f) for f in ("sbn.cu", "grouped.cu", "grads.cu", "adamw.cu")]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def _deps():
    files = list(SOURCES)
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            if f.endswith((".cuh", ".h", ".cu")):
                files.append(os.path.join(d, f))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def compile_command(src, out, ptxas_verbose=False):
    cmd = [
        NVCC, "-std=c++17", "-O3", "-lineinfo",
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
        "-c", src, "-o", out,
    ]
    if ptxas_verbose:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def link_command(objects, out):
    return [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "--cudart", "static",
            "-Xcompiler", "-fPIC", "-o", out] + objects


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libsbn.so next to this file (skipped when up to date). The
    sources compile side by side, in a scratch directory of this call."""
    if not force and up_to_date():
        return LIB
    with tempfile.TemporaryDirectory(prefix="sbn_build_") as tmp:
        objects = [os.path.join(tmp, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            logs = list(pool.map(lambda so: _run(compile_command(so[0], so[1], verbose)), zip(SOURCES, objects)))
        _run(link_command(objects, LIB + ".tmp"))
    if verbose:
        sys.stderr.write("".join(logs))
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
