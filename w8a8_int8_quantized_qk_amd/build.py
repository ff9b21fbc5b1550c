"""Build libqk.so (HIP, gfx950) in-tree with hipcc, and the Python module
_qkbind.so (host code only, torch's tensor interface) with g++.

Flags that matter for the numerics:
  -ffp-contract=off                       no multiply-add is fused unless the
                                          source writes fma
  -fhip-fp32-correctly-rounded-divide-sqrt binary32 '/' is the IEEE quotient
  -fno-gpu-flush-denormals-to-zero        binary32 subnormals are kept
  (no fast-math of any kind)
  -Xclang -target-feature -Xclang -packed-fp32-ops   no packed fp32 VALU ops
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libqk.so")
BIND = os.path.join(PKG, "_qkbind.so")
SOURCES = ["qk_api.hip", "quant.hip", "quant_static.hip", "gemm_mfma.hip", "gemm_wide.hip",
           "gemm_spec.hip", "gemm_slice.hip", "gemv.hip", "norm_quant.hip", "kv_cache.hip",
           "kv_attention.hip"]
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found: the HIP library cannot be built without ROCm")
    return path


def build_bind() -> str:
    """Compile csrc/bind.cpp against the installed torch, whose libraries the
    package has loaded by the time it imports the module."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    dirs = [*include_paths(), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for d in dirs for a in ("-isystem", d)],
           os.path.join(CSRC, "bind.cpp"), "-o", BIND + ".tmp",
           *["-L" + d for d in library_paths()], "-ltorch_python", "-ltorch_cpu", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{res.stderr}")
    os.replace(BIND + ".tmp", BIND)
    return BIND


def build(verbose: bool = False, jobs: int = 4) -> str:
    """Compile every HIP source for gfx950 and link libqk.so, and build
    _qkbind.so.  Always rebuilds."""
    cc = hipcc()
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed on {src}:\n{res.stderr}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        bind = ex.submit(build_bind)
        objs = list(ex.map(compile_one, SOURCES))
        bind.result()
    tmp = LIB + ".tmp"
    cmd = [cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
