"""Build the HIP library libmoe_ffn.so and the operators' call path
_opcall.so in-tree for gfx950.

Each source under csrc/ is compiled to an object under _build/ (in
parallel), then linked into moe_expert_ffn_persistent_amd/libmoe_ffn.so.
opcall.cpp is a Python module (host code against torch's headers); where it
cannot be built the library is, and the operators work without it.
Run ``python -m moe_expert_ffn_persistent_amd.build``; it always rebuilds.
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_ffn.so")
OPCALL = os.path.join(PKG, "_opcall.so")
ARCH = "gfx950"

SOURCES = ["layout.hip", "ffn_bf16.hip", "ffn_fp8.hip", "ffn_w4a8.hip", "combine.hip", "burst.hip",
           "mfma_probe.hip", "rows.hip", "swiglu.hip", "gemm_any.hip", "gemm_bf16.hip", "gemm_fp8.hip",
           "gemm_split.hip", "api.cpp", "ops_api.cpp", "planner.cpp"]

COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-I", INCLUDE, "-I", CSRC,
    # packed fp32 VALU ops stay off: hipcc emits them from plain float code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    # m0 is clobbered by the direct-to-LDS copies; the compiler keeps no value
    # of its own in m0 in these kernels
    "-Wno-inline-asm",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found: the HIP library cannot be built")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    if err.strip():
        print(err, file=sys.stderr)
    return obj


def _build_opcall() -> None:
    import torch

    root = os.path.dirname(torch.__file__)
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler found: the operators' call path cannot be built")
    tmp = OPCALL + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "opcall.cpp"), "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the C++ compiler failed for opcall.cpp:\n{r.stderr}")
    os.replace(tmp, OPCALL)


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES) + 1)) as ex:
        opcall = ex.submit(_build_opcall)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    try:
        opcall.result()
    except (RuntimeError, OSError, ImportError) as e:
        # the operators work without it; one of an earlier build may not fit
        if os.path.exists(OPCALL):
            os.remove(OPCALL)
        print(f"the operators' call path was not built, their calls will take longer: {e}", file=sys.stderr)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
