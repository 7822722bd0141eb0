"""Compiles the gfx950 HIP library libmoe_hip.so and the binding's native argument checks (_host.so) in-tree."""
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libmoe_hip.so")
HOST = os.path.join(PKG, "_host.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # each fp32 operation as written (bit-exact quantisation); FMAs are explicit
    "-ffp-contract=off",
    # no packed-fp32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.hip")))


def build(verbose: bool = False) -> str:
    cmd = [HIPCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc"),
           *sources(), "-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(LIB + ".tmp", LIB)
    try:
        build_host(verbose)
    except (OSError, subprocess.CalledProcessError, ImportError) as e:
        # optional, unlike the library: without the module (one of older
        # sources included) the Python checks run, a few microseconds a call slower
        if os.path.exists(HOST):
            os.remove(HOST)
        print(f"native argument checks not built ({e}); the Python ones run instead", file=sys.stderr, flush=True)
    return LIB


def build_host(verbose: bool = False) -> str:
    """csrc/host_checks.cpp: host code only, against torch's headers."""
    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in cpp_extension.include_paths()), f"-I{sysconfig.get_paths()['include']}",
           os.path.join(PKG, "csrc", "host_checks.cpp"), f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-o", HOST + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(HOST + ".tmp", HOST)
    return HOST


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
