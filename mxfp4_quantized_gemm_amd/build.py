"""Build libmxfp4.so (gfx950) in-tree with hipcc, and the torch binding of the
norm, 8-bit and attention operators (_ops.so, host code only) with g++.

Usage: python -m mxfp4_quantized_gemm_amd.build  (or build() from Python).
Every HIP source is compiled with -ffp-contract=off (the rotation butterfly
is an exact sequence of fp32 adds) and with packed-fp32 instructions
disabled. Objects go to _build/, the libraries next to this file.
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmxfp4.so")
OPS = os.path.join(PKG, "_ops.so")
SOURCES = ["api.cpp", "api_int8.cpp", "api_attention.cpp", "quant.hip", "gemm.hip", "stats.hip", "norm.hip",
           "int8_gemm.hip", "heads.hip", "attention.hip"]
OPS_SOURCES = ["torch_ops.cpp", "torch_attention.cpp"]
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libmxfp4)")


COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-Wall", "-Wno-unused-function",
]


def _compile(src: str) -> str:
    out = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc(), *COMMON, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = [ln for ln in (r.stderr or "").splitlines()
            if "not a recognized feature for this target" not in ln]
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n" + "\n".join(msgs))
    if msgs:
        sys.stderr.write("\n".join(msgs) + "\n")
    return out


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + r.stderr)


def _no_ops() -> str | None:
    """What the torch binding needs and this machine lacks, if anything."""
    if shutil.which("g++") is None:
        return "g++ is missing"
    try:
        import torch  # noqa: F401
        from torch.utils import cpp_extension
    except ImportError as e:
        return f"torch does not import ({e})"
    if not any(os.path.exists(os.path.join(d, "torch", "extension.h")) for d in cpp_extension.include_paths()):
        return "torch's headers are missing"
    return None


def _compile_ops() -> list[str]:
    """OPS_SOURCES -> objects: host code against torch's and HIP's headers."""
    with cf.ThreadPoolExecutor(max_workers=len(OPS_SOURCES)) as ex:
        return list(ex.map(_compile_ops_source, OPS_SOURCES))


def _compile_ops_source(src: str) -> str:
    import torch
    from torch.utils import cpp_extension
    out = os.path.join(BUILD, src + ".o")
    _run([shutil.which("g++"), "-O2", "-std=c++17", "-fPIC", "-c", "-D__HIP_PLATFORM_AMD__",
          "-DUSE_ROCM", "-DTORCH_EXTENSION_NAME=_ops", "-DTORCH_API_INCLUDE_EXTENSION_H",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *(f for d in [*cpp_extension.include_paths(), os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include"),
                        sysconfig.get_paths()["include"]] for f in ("-isystem", d)),
          os.path.join(CSRC, src), "-o", out], f"g++ on {src}")
    return out


def _link_ops(objs) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run([shutil.which("g++"), "-shared", "-o", OPS + ".tmp", *objs, "-L" + PKG, "-l:libmxfp4.so",
          "-L" + libs, "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch", "-ltorch_python",
          "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs], "linking _ops.so")
    os.replace(OPS + ".tmp", OPS)


def _link(objs) -> None:
    tmp = LIB + ".tmp"
    _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs], "linking libmxfp4.so")
    os.replace(tmp, LIB)


def build(verbose: bool = False) -> str:
    """Compile every source and link both libraries; returns libmxfp4.so's path.

    libmxfp4.so is linked first and needs nothing of the torch binding; on a
    machine without g++ or torch's headers it is built alone (the norm, 8-bit and attention
    modules then raise when they are imported)."""
    os.makedirs(BUILD, exist_ok=True)
    lacking = _no_ops()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ops = None if lacking else ex.submit(_compile_ops)
        _link(list(ex.map(_compile, SOURCES)))
        if ops:
            _link_ops(ops.result())
    if lacking:
        sys.stderr.write(f"_ops.so (norm, 8-bit and attention operators from Python) is not built: {lacking}\n")
        if os.path.exists(OPS):  # it may not fit the new library
            os.remove(OPS)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
