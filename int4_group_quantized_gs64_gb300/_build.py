"""Builds libqmv.so (the CUDA kernels and the C ABI) in-tree for sm_103a, and
_qmv_torch.so, the attention binding's argument checks for torch tensors.

Translation units are compiled in parallel with nvcc (the binding with g++)
and linked into one shared library next to this file; objects go to ``_build/``.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqmv.so")
TORCH_SRC = os.path.join(CSRC, "qmv_torch.cpp")
TORCH_LIB = os.path.join(HERE, "_qmv_torch.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-diag-suppress", "177"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqmv.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "qmv.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _torch_dir():
    spec = importlib.util.find_spec("torch")  # its place; torch itself is not imported to build
    return os.path.dirname(spec.origin) if spec else None


def _torch_up_to_date() -> bool:
    if _torch_dir() is None:
        return True
    return os.path.exists(TORCH_LIB) and all(
        os.path.getmtime(f) <= os.path.getmtime(TORCH_LIB)
        for f in (TORCH_SRC, os.path.join(INCLUDE, "qmv.h")))


def _torch_command(out):
    d = _torch_dir()
    inc = [os.path.join(d, "include"), os.path.join(d, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
           sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *("-I" + i for i in inc), TORCH_SRC,
            "-o", out, "-L" + os.path.join(d, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date() and _torch_up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    torch_tmp = None
    if force or not _torch_up_to_date():
        fd, torch_tmp = tempfile.mkstemp(suffix=".so", dir=HERE)
        os.close(fd)
        torch_cmd = _torch_command(torch_tmp)
        torch_proc = subprocess.Popen(torch_cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if force or not up_to_date():
        _build_lib(verbose)
    if torch_tmp:
        out, _ = torch_proc.communicate()
        if torch_proc.returncode:
            os.unlink(torch_tmp)
            raise RuntimeError("g++ failed:\n" + " ".join(torch_cmd) + "\n" + out.decode(errors="replace"))
        os.replace(torch_tmp, TORCH_LIB)
    return LIB


def _build_lib(verbose: bool) -> None:
    cc = nvcc()
    procs, objs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [cc, *NVCC_FLAGS, *ARCH, "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    errors = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            print(out.decode(errors="replace"))
        if p.returncode:
            errors.append(" ".join(cmd))
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=HERE)
    os.close(fd)
    subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
