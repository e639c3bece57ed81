"""Build libte_fp8.so (the gfx950 HIP kernels + the C ABI) and _te_ops.so (the Python side of the
operators around the GEMMs) in-tree."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libte_fp8.so")
BINDING = os.path.join(PKG, "_te_ops.so")
# (source, object, extra flags): gemm.hip is compiled once per operand-format pair and once for its
# host side (TE_GEMM_PART), so its kernel instantiations build in parallel
SOURCES = [("api.cpp", "api.o", []), ("api_ops.cpp", "api_ops.o", []), ("cast.hip", "cast.o", []),
           ("norm.hip", "norm.o", []), ("router.hip", "router.o", []), ("grad_clip.hip", "grad_clip.o", [])] + \
    [("gemm.hip", f"gemm_p{i}.o", [f"-DTE_GEMM_PART={i}"]) for i in range(9)]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
    # keep packed-fp32 VALU instructions out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _compile(job, verbose: bool) -> str:
    src, obj, extra = job
    obj = os.path.join(BUILD, obj)
    cmd = [HIPCC, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in (r.stderr or "").splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)
    return obj


def _build_binding(verbose: bool) -> str:
    """binding.cpp against PyTorch's headers and libraries (host code only)."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include"),
           *[f"-isystem{p}" for p in [*include_paths(), sysconfig.get_paths()["include"], "/opt/rocm/include"]],
           os.path.join(CSRC, "binding.cpp"), *[f"-L{p}" for p in library_paths()], "-ltorch_python", "-ltorch_cpu", "-ltorch_hip", "-lc10",
           "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_build_binding, verbose)
        objs = list(ex.map(lambda j: _compile(j, verbose), SOURCES))
        binding.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
