"""Build libdm0.so (the C-ABI library) in-tree for sm_100a with nvcc, and _language.so (the native binding of the
language operators, against the installed torch) with g++.

    python -m vla_dual_expert_b200.build [--force] [--ptxas-verbose]
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libdm0.so")
BINDING = os.path.join(HERE, "_language.so")
BINDING_STAMP = os.path.join(HERE, "_build", "language.stamp")
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(HERE, "csrc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def nvcc_path() -> str:
    return shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in _sources())


def _binding_sources():
    return [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "dm0.h")]


BINDING_FLAGS = ["-O2", "-std=c++20", "-fPIC", "-shared"]
BINDING_LIBS = ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]


def _binding_stamp() -> str:
    """What _language.so is built for: it uses the C++ internals of one torch and one interpreter."""
    return "\n".join([importlib.metadata.version("torch"), sysconfig.get_config_var("SOABI") or sys.version,
                      *BINDING_FLAGS, *BINDING_LIBS])


def _binding_fresh() -> bool:
    try:
        with open(BINDING_STAMP) as f:
            if f.read() != _binding_stamp():
                return False
        t = os.path.getmtime(BINDING)
    except OSError:
        return False
    return all(os.path.getmtime(s) <= t for s in _binding_sources())


def build_binding(force: bool = False) -> str:
    """_language.so; needs libdm0.so, which it links against (found beside it)."""
    if not force and _binding_fresh():
        return BINDING
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    cmd = [shutil.which("g++") or "g++", *BINDING_FLAGS,
           "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"], "-I", INCLUDE,
           os.path.join(CSRC, "binding.cpp"), "-o", BINDING + ".tmp",
           "-L" + os.path.join(torch, "lib"), *BINDING_LIBS,
           "-L" + HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(BINDING + ".tmp", BINDING)
    os.makedirs(os.path.dirname(BINDING_STAMP), exist_ok=True)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_stamp())
    return BINDING


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    build_library(force, ptxas_verbose)
    if importlib.util.find_spec("torch"):   # the language operators take its tensors; all else runs without it
        build_binding(force)
    return LIB


def build_library(force: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    cmd = [nvcc_path(), "-O3", "-std=c++17",
           "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
           "-Xcompiler", "-fPIC", "-shared", "--expt-relaxed-constexpr",
           "-I", INCLUDE, "-I", CSRC,
           "-o", LIB + ".tmp", os.path.join(CSRC, "dm0.cu")]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if ptxas_verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, ptxas_verbose="--ptxas-verbose" in sys.argv)
    print(LIB)
