"""Ahead-of-time build of librz_fp8.so for gfx950 (hipcc, in-tree) and, as a
step of its own, of the binding's native half (g++, against torch and that
library).

The library is the product: HIP kernels plus the C ABI declared in
include/rz_fp8.h.  It is compiled for gfx950 only, without fast-math, with
floating-point contraction off and IEEE fp32 division, and with packed fp32
instructions disabled.  It needs neither Python's nor torch's headers.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_NAME = "librz_fp8.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
SOURCES = ["api.hip", "kquant.hip", "actquant.hip", "gemm.hip", "gemm_edge.hip", "kgemv.hip", "kqgemm.hip",
           "q8gemm.hip", "mxquant.hip", "mxgemm.hip", "mxgemv.hip", "kvcache.hip",
           "kvplan.hip", "kvattn.hip", "kvselect.hip"]
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-ffp-contract=off",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-parallel-jobs=8",  # one source each
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cand = os.path.join(rocm, "bin", "hipcc")
    return cand if os.path.exists(cand) else "hipcc"


def build(verbose: bool = False) -> str:
    """Compile every HIP source into LIB_PATH (always rebuilds)."""
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    tmp = LIB_PATH + ".tmp"
    cmd = [hipcc(), *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), *srcs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature name: drop that noise
    noise = ("unknown target feature", "packed-fp32-ops")
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if not any(n in ln for n in noise)]
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs), flush=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def native_path() -> str:
    """The native half's file, named after the torch and Python it is built
    against: another one's copy is not found rather than loaded."""
    torch = importlib.metadata.version("torch")
    return os.path.join(PKG_DIR, f"_rz_native.torch-{torch}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_native(verbose: bool = False) -> str:
    """csrc/native.cpp -> native_path(), linked to the library beside it."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("the binding's native half is built against torch, which is not installed")
    torch_dir = os.path.dirname(spec.origin)
    path = native_path()
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    tmp = path + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(rocm, "include"), "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "native.cpp"), "-o", tmp,
           "-L", PKG_DIR, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, path)
    return path


def build_all(verbose: bool = False) -> list[str]:
    """The library and, where torch is installed, the binding's native half."""
    made = [build(verbose)]
    if importlib.util.find_spec("torch") is None:
        print("torch is not installed: the binding's native half is left out", file=sys.stderr, flush=True)
    else:
        made.append(build_native(verbose))
    return made


if __name__ == "__main__":
    print("\n".join(build_all(verbose="-v" in sys.argv)))
