"""Builds the in-tree shared libraries with nvcc for sm_100a.

  libmoe_nvfp4.so   the MoE layer (csrc/*.cu, C ABI in include/moe_nvfp4.h)
  libmoe_inputs.so  the device writer of synthetic banks (moe_inputs/fill.cu)

Usage: python -m nvfp4_weight_only_top_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmoe_nvfp4.so")
INPUTS_SRC = os.path.join(ROOT, "moe_inputs", "fill.cu")
INPUTS_LIB = os.path.join(ROOT, "moe_inputs", "libmoe_inputs.so")

# Sources compiled on their own, which share no device symbols with the others: in relocatable device code
# setmaxnreg (a register split between warps, fp8_matmul.cu) is ignored, and a kernel that calls a function that
# is not inlined gets the registers that the function would like (route_scored.cu: 110, where its launch bounds
# leave 64; fp8_quant.cu).
WHOLE = {"fp8_matmul.cu", "fp8_quant.cu", "route_scored.cu"}

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(out: str, deps: list) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd: list, verbose: bool) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"nvcc failed ({r.returncode}): {' '.join(cmd)}")
    if verbose:
        sys.stdout.write(r.stdout + r.stderr)
    return " ".join(cmd) + "\n" + r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False) -> list:
    """Compiles both libraries if their sources changed; returns the library paths."""
    nvcc = _nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h"))
    if force or _stale(LIB, deps):
        tmp = LIB + ".tmp"
        with tempfile.TemporaryDirectory() as objs:
            def compile_one(src):
                name = os.path.basename(src)
                obj = os.path.join(objs, name[:-3] + ".o")
                rdc = [] if name in WHOLE else ["-rdc=true"]
                return obj, _run([nvcc, *ARCH, *FLAGS, *rdc, "-I", INCLUDE, "-c", "-o", obj, src], verbose)
            with concurrent.futures.ThreadPoolExecutor(os.cpu_count() or 1) as pool:
                done = list(pool.map(compile_one, srcs))
            log = "".join(text for _, text in done)
            log += _run([nvcc, *ARCH, *FLAGS, "-shared", "-rdc=true", "-o", tmp, *(o for o, _ in done)], verbose)
        with open(os.path.join(PKG, "build_moe_nvfp4.log"), "w") as f:
            f.write(log)
        os.replace(tmp, LIB)
    if force or _stale(INPUTS_LIB, [INPUTS_SRC]):
        tmp = INPUTS_LIB + ".tmp"
        with open(os.path.join(PKG, "build_moe_inputs.log"), "w") as f:
            f.write(_run([nvcc, *ARCH, *FLAGS, "-shared", "-o", tmp, INPUTS_SRC], verbose))
        os.replace(tmp, INPUTS_LIB)
    return [LIB, INPUTS_LIB]


if __name__ == "__main__":
    print("\n".join(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)))
