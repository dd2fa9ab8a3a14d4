"""Build libkq.so (the CUDA kernels and the C ABI) in-tree for sm_100a, and
_calls.so (the binding's fast path) against the installed torch, where that
has its headers and there is a g++.

    python -m dequant_quant_gemv_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libkq.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "kq_calls.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + [os.path.join(ROOT, "include", "kq.h")])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


FLAGS = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include")]


def calls_key() -> str:
    """What _calls.so is built against: another torch, C++ ABI or Python needs another one."""
    import sysconfig

    import torch
    return f"{torch.__version__} {int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('SOABI')}"


def _calls_dirs() -> tuple[list[str], str]:
    """Where _calls.so's headers and libraries are."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    cuda = os.path.dirname(os.path.dirname(NVCC))
    return ([*include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")],
            os.path.join(os.path.dirname(torch.__file__), "lib"))


def _calls_lack() -> str | None:
    """What _calls.so needs and is not there."""
    inc, lib = _calls_dirs()
    for header in ("torch/csrc/autograd/python_variable.h", "c10/cuda/CUDAStream.h", "Python.h", "cuda_runtime_api.h"):
        if not any(os.path.exists(os.path.join(d, header)) for d in inc):
            return header
    for so in ("libtorch_python.so", "libc10_cuda.so"):
        if not os.path.exists(os.path.join(lib, so)):
            return so
    return None if shutil.which("g++") else "g++"


def _calls_command(out: str) -> list[str]:
    import torch
    inc, lib = _calls_dirs()
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DKQ_CALLS_KEY="{calls_key()}"',
            *[x for d in inc for x in ("-isystem", d)], "-o", out, CALLS_SRC,
            f"-L{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _calls_current() -> bool:
    """Whether _calls.so is newer than its sources and built against this torch and Python."""
    if not os.path.exists(CALLS):
        return False
    newest = max(os.path.getmtime(f) for f in (CALLS_SRC, os.path.join(ROOT, "include", "kq.h"), os.path.abspath(__file__)))
    with open(CALLS, "rb") as f:
        return os.path.getmtime(CALLS) >= newest and calls_key().encode() + b"\0" in f.read()


def build_calls(force: bool = False):
    """Start building _calls.so where it is out of date: (process, temporary file), or None."""
    if not force and _calls_current():
        return None
    lack = _calls_lack()
    if lack:  # (the binding calls through ctypes then; a compilation that fails is an error)
        print(f"_calls.so is not built: no {lack}")
        return None
    tmp = CALLS + f".tmp{os.getpid()}"
    return subprocess.Popen(_calls_command(tmp), stdout=subprocess.PIPE, stderr=subprocess.STDOUT), tmp


def finish_calls(started) -> None:
    if started is None:
        return
    p, tmp = started
    out, _ = p.communicate()
    if p.returncode:
        sys.stdout.write(out.decode(errors="replace"))
        if os.path.exists(tmp):
            os.remove(tmp)
        raise RuntimeError("g++ failed for kq_calls.cpp")
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """Compile every csrc/*.cu to an object (in parallel), link libkq.so, and build _calls.so."""
    calls = build_calls(force)
    try:
        if force or not up_to_date():
            _build_lib(verbose)
    finally:
        finish_calls(calls)
    return LIB


def _build_lib(verbose: bool) -> None:
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    procs, objs = [], []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [NVCC, *FLAGS, "-c", "-o", obj, src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            sys.stdout.write(out.decode(errors="replace"))
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, *ARCH, "--shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
