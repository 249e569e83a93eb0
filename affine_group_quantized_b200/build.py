"""Build libqmv.so (the sm_100a kernels and the C ABI) in-tree with nvcc, and
the CPython module of the binding's kv_* calls with the host compiler.

The library is compiled for sm_100a only.  It is placed next to this file so
that it travels with the repository and is the one the Python binding loads.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libqmv.so")
NATIVE = os.path.join(HERE, "_kv_native" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["qmv_api.cu", "qmv_quant.cu", "qmv_qmm.cu", "qmv_kv.cu", "qmv_kv_attn4.cu",
           "qmv_kv_attn8.cu", "qmv_kv_attn16.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CC = os.environ.get("CC", "gcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-warn-spills",
]


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "qmv.h"))
    return files


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB) and os.path.exists(NATIVE):
        newest = max(os.path.getmtime(f) for f in _inputs())
        if min(os.path.getmtime(LIB), os.path.getmtime(NATIVE)) >= newest:
            return LIB
    # one object per source, compiled side by side, then one link
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    procs, objs = [], []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [NVCC, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj,
               os.path.join(CSRC, src)]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        procs.append((src, subprocess.Popen(cmd)))
        objs.append(obj)
    failed = [src for src, pr in procs if pr.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, "nvcc " + " ".join(failed))
    link = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
            "-o", LIB + ".tmp", *objs]
    subprocess.run(link, check=True)
    os.replace(LIB + ".tmp", LIB)
    # the module calls libqmv.so, found beside it
    subprocess.run([CC, "-O2", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"],
                    "-I", INCLUDE, "-o", NATIVE + ".tmp", os.path.join(CSRC, "kv_native.c"),
                    "-L", HERE, "-l:libqmv.so", "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(NATIVE + ".tmp", NATIVE)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
