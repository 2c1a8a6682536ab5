"""Build libmoe_gb300.so in-tree with nvcc for sm_103a (GB300) only, and beside it the torch
marshalling of the operators around the experts (block_binding.cpp, host code) with g++."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmoe_gb300.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(ROOT, "include", "moe_gb300.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in deps())


BINDING_SRC = os.path.join(CSRC, "binding", "block_binding.cpp")


def binding_path() -> str:
    """The marshalling extension for the installed torch (it uses torch's C++ headers, so a file per version)."""
    import torch

    return os.path.join(PKG, "_block_ext_" + "".join(c if c.isalnum() else "_" for c in torch.__version__) + ".so")


def binding_up_to_date() -> bool:
    path = binding_path()
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path)
                                        for p in (BINDING_SRC, os.path.join(ROOT, "include", "moe_gb300.h")))


def _start_binding():
    """Start g++ on the extension; returns (process, temporary output, final path)."""
    import sysconfig

    import torch

    path = binding_path()
    tmp = path + f".tmp{os.getpid()}"
    home = os.path.dirname(torch.__file__)
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{i}" for i in inc], BINDING_SRC, "-o", tmp, "-L" + os.path.join(home, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), tmp, path


def _finish_binding(started) -> str:
    proc, tmp, path = started
    out = proc.communicate()[0]
    if proc.returncode != 0:
        sys.stderr.write(out)
        raise RuntimeError("g++ failed building the torch binding of the operators around the experts")
    os.replace(tmp, path)
    return path


def build_binding() -> str:
    return binding_path() if binding_up_to_date() else _finish_binding(_start_binding())


def build_all(force: bool = False) -> None:
    """The library and the binding, compiled side by side."""
    started = _start_binding() if force or not binding_up_to_date() else None
    try:
        build(force)
    finally:
        if started is not None:
            _finish_binding(started)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-lineinfo", *ARCH,
           "--threads", "0", "-I", os.path.join(ROOT, "include"), "-o", tmp, *sources()]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc failed building libmoe_gb300.so")
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
