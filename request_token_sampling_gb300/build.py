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
    "strata_kernel.cuh", "strata_device.cuh", "strata_resident.cuh", "strata_merge.cuh", "strata_host.h", "strata_chain.h",
    "strata_norm.cuh", "strata_draw.cuh", "strata_project.cuh")]
DEPENDS += [os.path.join(ROOT, "include", f) for f in ("strata_sample.h", "strata_tail.h")]
MODULE_PATH = os.path.join(LIB_DIR, "_strata_tail.so")
MODULE_SOURCE = os.path.join(CSRC, "tail_binding.cpp")
DEPENDS += [MODULE_SOURCE]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(MODULE_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(MODULE_PATH))
    return all(os.path.getmtime(p) <= t for p in DEPENDS)


def module_commands(out: str):
    """Compile and link the PyTorch binding (host code only) against the installed PyTorch and Python."""
    import sysconfig
    from importlib.util import find_spec
    torch_dir = os.path.dirname(find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    obj = os.path.join(LIB_DIR, "tail_binding.o")
    libs = os.path.join(torch_dir, "lib")
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *[f for d in inc for f in ("-isystem", d)], "-c", "-o",
                obj, MODULE_SOURCE]
    link = ["g++", "-shared", "-o", out, obj, "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
            "-lc10_cuda", "-lc10", "-L" + LIB_DIR, "-l:" + os.path.basename(LIB_PATH), "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/ into _lib/: libstrata_sample.so (statically linked CUDA runtime) and the PyTorch binding."""
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
    compile_module, link_module = module_commands(MODULE_PATH + ".tmp")
    started.append(subprocess.Popen(compile_module, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    said = [p.communicate()[0] for p in started]
    for p, text in zip(started, said):
        if p.returncode != 0:
            raise RuntimeError(f"{p.args[0]} failed:\n" + text)
        if verbose:
            print(text)
    r = subprocess.run([nvcc_path(), *ARCH_FLAGS, "-shared", "-o", tmp, *objects], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed to link:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB_PATH)
    r = subprocess.run(link_module, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed to link:\n" + r.stdout + r.stderr)
    os.replace(MODULE_PATH + ".tmp", MODULE_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build_library(force=True, verbose=True)
