"""Build libbq.so (the CUDA library behind include/bq.h) in-tree with nvcc for
sm_100a, and, where torch is installed, the binding's compiled calls on torch tensors
(_torch_calls.so).  Usage: python -m block_scaled_precision_quant_b200.build [--force]"""
from __future__ import annotations

import contextlib
import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbq.so")
CALLS = os.path.join(PKG, "_torch_calls.so")
CALLS_STAMP = os.path.join(PKG, "_torch_calls.built")
CALLS_SOURCE = os.path.join(CSRC, "torch_calls.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC",
    "-Xptxas", "-v", "--threads", "0",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def current(built: str, files) -> bool:
    if not os.path.exists(built):
        return False
    t = os.path.getmtime(built)
    return all(os.path.getmtime(d) <= t for d in files)


def up_to_date() -> bool:
    return current(LIB, deps())


def built_for() -> str:
    """The interpreter and the torch whose C++ interfaces the compiled calls are built against."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "?"
    return f"{sysconfig.get_config_var('SOABI')} torch {torch}"


def calls_built_for():
    """built_for() of the build of the compiled calls at hand, None if it is not known."""
    try:
        with open(CALLS_STAMP) as f:
            return f.read()
    except OSError:
        return None


def build_calls(force: bool = False):
    """The extension module of csrc/torch_calls.cpp (g++), or None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    if (not force and calls_built_for() == built_for()
            and current(CALLS, [CALLS_SOURCE, os.path.join(INCLUDE, "bq.h")])):
        return CALLS
    torch_dir = os.path.dirname(spec.origin)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    with contextlib.suppress(FileNotFoundError):
        os.remove(CALLS)  # of other sources: not to be loaded should this build fail
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden", "-I", INCLUDE, "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(cuda, "include"), CALLS_SOURCE,
           "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed building _torch_calls.so")
    os.replace(tmp, CALLS)
    with open(CALLS_STAMP, "w") as f:
        f.write(built_for())
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    build_lib(force, verbose)
    try:
        build_calls(force)
    except (RuntimeError, OSError) as e:  # the library does without; what needs them says so
        warnings.warn(f"the binding's compiled calls are not built: {e}")
    return LIB


def build_lib(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, *sources(), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    log = r.stdout + r.stderr
    with open(os.path.join(PKG, "build.log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + log)
    if r.returncode != 0:
        sys.stderr.write(log)
        raise RuntimeError("nvcc failed building libbq.so (see block_scaled_precision_quant_b200/build.log)")
    if verbose:
        sys.stderr.write(log)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
