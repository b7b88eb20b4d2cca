"""Builds libssm.so (the HIP kernels and the C ABI) in-tree with hipcc for gfx950,
and _marshal.so (host code of the Python binding) with g++."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libssm.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
SOURCES = ["ssm_abi.cpp", "scan_fwd.hip", "scan_bwd.hip", "ssd_fwd.hip", "ssd_bwd.hip", "update_fwd.hip",
           "conv_fwd.hip", "layer_abi.cpp", "gated_scan.hip", "rms_norm.hip", "w4_matvec.hip"]
HEADERS = ["ssm_internal.h", "layer_internal.h", "abi_checks.h", "column_sums.h", "w4_loads.h",
           os.path.join("..", "..", "include", "ssm.h")]

# Packed fp32 VALU ops are kept out of all device code.
HIPCC_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared", "-Wall",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build_marshal() -> str:
    """Compile marshal.cpp, a CPython module over torch's tensors (host code only)."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    inc = os.path.join(root, "include")
    tmp = MARSHAL + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I", sysconfig.get_path("include"), "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           os.path.join(CSRC, "marshal.cpp"), "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-o", tmp]
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout)
    os.replace(tmp, MARSHAL)
    return MARSHAL


def build(verbose: bool = False) -> str:
    """Compile every source into libssm.so and _marshal.so (always recompiles)."""
    build_marshal()
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [hipcc()] + HIPCC_FLAGS + ["-I", os.path.join(HERE, "..", "include")] + srcs + ["-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so; that is harmless.
    out = "\n".join(l for l in res.stdout.splitlines() if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + out)
    if verbose and out.strip():
        print(out, file=sys.stderr)
    os.replace(tmp, LIB)
    return LIB


def needs_build() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS + ["marshal.cpp"]]
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


if __name__ == "__main__":
    print(build(verbose=True))
