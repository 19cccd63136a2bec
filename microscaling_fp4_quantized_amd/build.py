"""Build libfp4.so (the HIP library behind include/fp4.h) for gfx950 with hipcc.

Usage: python -m microscaling_fp4_quantized_amd.build   (or build() from Python)

Compiles every source under csrc/ to an object in _build/ (in parallel) and links
the shared library next to this file, and with it _torch_calls.so, the host-only
module that enters the library from torch tensors. Always recompiles. The library
needs hipcc alone; without a host compiler, Python's headers or torch the module is
left out, with a warning, and binding.py marshals every call itself.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfp4.so")
CALLS = os.path.join(HERE, "_torch_calls.so")

SOURCES = [
    "rotate_quant.hip",
    "gemm_mxfp4.hip",
    "gemm_mxfp4_ring.hip",
    "gemm_decode.hip",
    "gemm_nvfp4.hip",
    "gemm_nvfp4_ring.hip",
    "fp8_quant.hip",
    "gemm_fp8_split.hip",
    "gemm_fp8_ring.hip",
    "moe.hip",
    "fp4_abi.cpp",
]

ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fvisibility=hidden",
    # the rotation is specified operation by operation: no contraction into FMAs
    "-ffp-contract=off",
    # IEEE float32 subnormals (the rotation and the scale rules depend on them)
    "-fno-gpu-flush-denormals-to-zero",
    # no packed float32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    f"-I{os.path.join(ROOT, 'include')}",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj] + FLAGS
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{out}")
    if out.strip():
        print(out, file=sys.stderr)
    return obj


def _build_calls() -> str:
    """_torch_calls.so against the installed torch's headers (host code only)."""
    import torch
    from torch.utils import cpp_extension

    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no host C++ compiler found")
    tmp = CALLS + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{d}" for d in cpp_extension.include_paths()), f"-isystem{sysconfig.get_paths()['include']}",
           os.path.join(CSRC, "torch_calls.cpp"), "-o", tmp,
           *(f"-L{d}" for d in cpp_extension.library_paths()), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"host compiler failed on torch_calls.cpp:\n{r.stdout}{r.stderr}")
    os.replace(tmp, CALLS)
    return CALLS


def _link(objs) -> None:
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=5) as ex:
        calls = ex.submit(_build_calls)
        _link(list(ex.map(_compile, SOURCES)))
        try:
            calls.result()
            module = f" and {os.path.basename(CALLS)}"
        except Exception as e:  # whatever the host lacks: the library stands without it
            module = ""
            if os.path.exists(CALLS):
                os.remove(CALLS)  # one of an earlier build was compiled for another library
            print(f"warning: {os.path.basename(CALLS)} not built, Python calls take longer: {e}", file=sys.stderr)
    if verbose:
        print(f"built {LIB}{module}")
    return LIB


if __name__ == "__main__":
    build()
