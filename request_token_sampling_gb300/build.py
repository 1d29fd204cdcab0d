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


def torch_dir() -> str | None:
    """Where PyTorch is installed, if it is (it is not imported)."""
    from importlib.util import find_spec
    spec = find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def up_to_date() -> bool:
    made = [LIB_PATH] + ([MODULE_PATH] if torch_dir() else [])
    if not all(os.path.exists(p) for p in made):
        return False
    t = min(os.path.getmtime(p) for p in made)
    return all(os.path.getmtime(p) <= t for p in DEPENDS)


def module_commands(out: str, torch: str):
    """Compile and link the PyTorch binding (host code only) against the PyTorch in `torch` and this Python."""
    import sysconfig
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    obj = os.path.join(LIB_DIR, "tail_binding.o")
    libs = os.path.join(torch, "lib")
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *[f for d in inc for f in ("-isystem", d)], "-c", "-o",
                obj, MODULE_SOURCE]
    link = ["g++", "-shared", "-o", out, obj, "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
            "-lc10_cuda", "-lc10", "-L" + LIB_DIR, "-l:" + os.path.basename(LIB_PATH), "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/ into _lib/: libstrata_sample.so (statically linked CUDA runtime) and, where PyTorch is
    installed, the operators' PyTorch binding."""
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
    torch = torch_dir()
    if torch:
        compile_module, link_module = module_commands(MODULE_PATH + ".tmp", torch)
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
    if torch:
        r = subprocess.run(link_module, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("g++ failed to link:\n" + r.stdout + r.stderr)
        os.replace(MODULE_PATH + ".tmp", MODULE_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build_library(force=True, verbose=True)
