"""Build the sampler's shared library in-tree with nvcc for sm_103a (no cmake; its files compile side by side)."""
from __future__ import annotations

import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libstrata_sample.so")
SOURCES = [os.path.join(CSRC, f) for f in ("strata_sample.cu", "strata_tail.cu", "strata_project.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in (
    "strata_kernel.cuh", "strata_device.cuh", "strata_resident.cuh", "strata_merge.cuh", "strata_host.h",
    "strata_norm.cuh", "strata_draw.cuh", "strata_project.cuh")]
DEPENDS += [os.path.join(ROOT, "include", f) for f in ("strata_sample.h", "strata_tail.h")]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in DEPENDS)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/ into _lib/libstrata_sample.so (statically linked CUDA runtime)."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB_PATH + ".tmp"
    flags = [*ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags.append("-Xptxas=-v")
    objects = [os.path.join(LIB_DIR, os.path.splitext(os.path.basename(s))[0] + ".o") for s in SOURCES]
    started = [subprocess.Popen([nvcc_path(), *flags, "-c", "-o", o, s], stdout=subprocess.PIPE,
                                stderr=subprocess.STDOUT, text=True) for s, o in zip(SOURCES, objects)]
    said = [p.communicate()[0] for p in started]
    for p, text in zip(started, said):
        if p.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + text)
        if verbose:
            print(text)
    r = subprocess.run([nvcc_path(), *ARCH_FLAGS, "-shared", "-o", tmp, *objects], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed to link:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build_library(force=True, verbose=True)
