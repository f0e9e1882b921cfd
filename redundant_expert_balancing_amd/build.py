"""Build libmoonep.so (HIP, gfx950) and the compiled part of its Python binding in-tree:
``python -m redundant_expert_balancing_amd.build``."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libmoonep.so")
BINDING = os.path.join(PKG, "_binding.so")

HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # never let the compiler emit packed fp32 arithmetic
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.hip")))


def _hipcc() -> str:
    return os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def _host_compiler() -> str:
    """CXX, or g++ where there is one, or the C++ compiler beside hipcc."""
    return (os.environ.get("CXX") or shutil.which("g++")
            or os.path.join(os.path.dirname(_hipcc()), "amdclang++"))


def build_library(verbose: bool = False) -> str:
    """Compile every HIP source into libmoonep.so next to this file; return its path."""
    hipcc = _hipcc()
    tmp = LIB + ".tmp"
    cmd = [hipcc, *HIP_FLAGS, "-I", os.path.join(ROOT, "include"), *sources(), "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)
    os.replace(tmp, LIB)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """Compile csrc/binding.cpp (host code) against torch's headers; return its path."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    inc = os.path.join(base, "include")
    tmp = BINDING + ".tmp"
    cmd = [_host_compiler(), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"], "-I", inc,
           "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           os.path.join(PKG, "csrc", "binding.cpp"), "-o", tmp,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding's compiler failed ({res.returncode}):\n{res.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build_library(verbose=True))
    print(build_binding(verbose=True))
