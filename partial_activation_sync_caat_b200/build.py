"""Builds libcaat.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m partial_activation_sync_caat_b200.build [--verbose-ptxas]

The library links the CUDA runtime statically, fetches the driver's tensor-map encoder at
run time, and so loads on a machine without a GPU (the ABI tests rely on that).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libcaat.so")

SOURCES = ["caat_api.cu", "attn_api.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    files = [os.path.join(INCLUDE, "caat.h")]
    for f in os.listdir(CSRC):
        if f.endswith((".cu", ".cuh", ".h")):
            files.append(os.path.join(CSRC, f))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not verbose_ptxas and up_to_date():
        return LIB
    tmp = LIB + ".tmp"
    base = [nvcc_path(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
            "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC, "-DCAAT_BUILD"]
    if verbose_ptxas:
        base.insert(1, "-Xptxas=-v")
    with tempfile.TemporaryDirectory() as objs:  # the sources compile side by side, then link
        jobs = []
        for src in SOURCES:
            cmd = base + ["-c", os.path.join(CSRC, src), "-o", os.path.join(objs, src + ".o")]
            jobs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        outs = [(cmd, p.communicate()[0], p.returncode) for cmd, p in jobs]
        if all(rc == 0 for _, _, rc in outs):
            cmd = base + ["-shared", "-o", tmp] + [os.path.join(objs, src + ".o") for src in SOURCES]
            res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            outs.append((cmd, res.stdout, res.returncode))
    for cmd, text, rc in outs:
        if rc != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + text)
        if verbose_ptxas:
            sys.stderr.write(text)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="--verbose-ptxas" in sys.argv))
