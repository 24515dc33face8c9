"""Builds libcaat.so (the C-ABI library) in-tree with nvcc for sm_100a, and _marshal-*.so (the compiled
half of the Python binding, against PyTorch's headers) with g++.

    python -m partial_activation_sync_caat_b200.build [--verbose-ptxas]

The library links the CUDA runtime statically, fetches the driver's tensor-map encoder at
run time, and so loads on a machine without a GPU (the ABI tests rely on that).
"""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from typing import Optional

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


def torch_version() -> Optional[str]:
    """The installed PyTorch's version, read from its files (importing it takes seconds); None without one."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        return re.search(r"^__version__ = ['\"](.+)['\"]", f.read(), re.M).group(1)


def marshal_path(version: Optional[str] = None) -> str:
    """The compiled marshalling for a PyTorch version (default: the installed one) and this interpreter.  It
    reads their objects by the layouts that it was compiled for, so the name says which: under any other, there
    is no such file."""
    return os.path.join(PKG, f"_marshal-torch{version or torch_version()}-{sysconfig.get_config_var('SOABI')}.so")


def _newer(out: str, endings) -> bool:
    files = [os.path.join(INCLUDE, "caat.h")] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(endings)]
    return os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out) for f in files)


def up_to_date() -> bool:
    """Whether the library is (what the binding can do without is not asked for)."""
    return _newer(LIB, (".cu", ".cuh", ".h"))


def marshal_up_to_date() -> bool:
    return torch_version() is None or _newer(marshal_path(), (".cpp",))


def _marshal_command(out: str) -> list:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    system = [os.path.join(torch, "include"), sysconfig.get_paths()["include"], cuda]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            *(x for d in system for x in ("-isystem", d)), "-I", INCLUDE, os.path.join(CSRC, "marshal.cpp"), "-o", out,
            "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _start(cmd):
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _start_marshal():
    """Starts the compiler on the compiled marshalling and returns what finishes it.  The binding can do without
    (its calls then take the host longer), so no failure of this stops the library's build; a file of older
    sources goes, since the structures of its calls may be others."""
    if torch_version() is None:
        return lambda: None
    path = marshal_path()
    cmd, job, why = [], None, ""
    try:
        cmd = _marshal_command(path + ".tmp")
        job = _start(cmd)
    except (OSError, RuntimeError) as e:
        why = str(e)

    def finish():
        text = job.communicate()[0] if job else why
        if job and job.returncode == 0:
            os.replace(path + ".tmp", path)
            return
        for f in (path + ".tmp", path):
            if os.path.exists(f):
                os.remove(f)
        sys.stderr.write("the compiled marshalling was not built; calls will be marshalled in Python:\n"
                         + " ".join(cmd) + "\n" + text + "\n")
    return finish


def _build_library(verbose_ptxas: bool):
    tmp = LIB + ".tmp"
    base = [nvcc_path(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
            "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC, "-DCAAT_BUILD"]
    if verbose_ptxas:
        base.insert(1, "-Xptxas=-v")
    with tempfile.TemporaryDirectory() as objs:  # the sources compile side by side, then link
        jobs = []
        for src in SOURCES:
            cmd = base + ["-c", os.path.join(CSRC, src), "-o", os.path.join(objs, src + ".o")]
            jobs.append((cmd, _start(cmd)))
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
    return tmp


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    force = force or verbose_ptxas
    finish = _start_marshal() if force or not marshal_up_to_date() else lambda: None
    try:
        tmp = _build_library(verbose_ptxas) if force or not up_to_date() else None
    finally:
        finish()
    if tmp:  # last: whoever waits for the library finds the marshalling beside it
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="--verbose-ptxas" in sys.argv))
