"""Builds libssm_gb300.so in-tree: every .cu under csrc/ compiled for sm_103a only.

Usage: ``python -m bwd_ssm_conv_gb300.build`` (or ``build()`` from Python).  Objects are
compiled in parallel; the library links the shared CUDA runtime so that it and PyTorch use
one runtime instance in a process.  Beside it goes _block.so, the Python module that marshals the
calls of ssm_block.h: host code against PyTorch's headers.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libssm_gb300.so")
MODULE = os.path.join(HERE, "_block.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libssm_gb300.so")


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def _torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _module_source() -> str:
    return os.path.join(CSRC, "block_binding.cpp")


def _compile_module(nvcc: str) -> str:
    """The module's object; a C++ compiler, as it holds no device code."""
    obj = os.path.join(BUILD_DIR, "block_binding.o")
    torch_include = os.path.join(_torch_dir(), "include")
    cuda_include = os.path.join(os.path.dirname(_cuda_lib_dir(nvcc)), "include")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE,
          "-isystem", torch_include,
          "-isystem", os.path.join(torch_include, "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda_include,
          "-c", _module_source(), "-o", obj])
    return obj


def _link_module(obj: str) -> None:
    tmp = MODULE + f".{os.getpid()}.tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", HERE,
          "-l:" + os.path.basename(LIB), "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python",
          "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, MODULE)


def _run(cmd) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{' '.join(cmd)} failed:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MODULE):
        return False
    t, m = os.path.getmtime(LIB), os.path.getmtime(MODULE)
    # the module also goes with the PyTorch that it was compiled against
    torch_version = os.path.join(_torch_dir(), "version.py")
    return (all(os.path.getmtime(p) <= t for p in _deps()) and
            all(os.path.getmtime(p) <= m for p in [LIB, _module_source(), torch_version]))


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not ptxas_info and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        module = ex.submit(_compile_module, nvcc)
        results = list(ex.map(compile_one, _sources()))
    if verbose or ptxas_info:
        for _, err in results:
            if err:
                sys.stderr.write(err)
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *[o for o, _ in results],
           "-Xlinker", f"-rpath,{_cuda_lib_dir(nvcc)}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_module(module.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
