"""Compile the HIP library in-tree for gfx950: ``python -m mixture_experts_expert_histogram_amd.build``."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB_NAME = "libmoe_mi355x.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
SOURCES = ["route.hip", "gemm.hip", "gemm_dma.hip", "gemm_mx.hip", "few.hip", "mx.hip", "ffn_fwd.hip",
           "ffn_bwd.hip", "ffn_few.hip", "norm.hip", "ortho.hip", "api.cpp", "api_block.cpp"]
BINDING, BINDING_NAME = "binding.cpp", "_block.so"   # the native half of the Python binding
ARCH = "gfx950"


def hipcc() -> str:
    for c in [os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")]:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build the MoE library)")


def compile_flags():
    return ["-x", "hip", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"), "-Wno-unused-result", "-Wno-inline-asm"]


def binding_commands(obj: str, out: str):
    """g++ on the CPython module of the operators around the routed experts (torch's headers and libraries): compile, link."""
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-c", os.path.join(CSRC, BINDING), "-o", obj,
             "-I", os.path.join(t, "include"), "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
             "-I", sysconfig.get_paths()["include"], "-I", os.path.join(rocm, "include")],
            ["g++", "-shared", obj, "-o", out, "-L", os.path.join(t, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python",
             "-Wl,-rpath," + os.path.join(t, "lib"), LIB_PATH, "-Wl,-rpath,$ORIGIN"])


def run_all(what: str, jobs, verbose: bool = False) -> None:
    """Run the commands of jobs [(name, command)] side by side; RuntimeError names those that fail."""
    procs = []
    for name, cmd in jobs:
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((name, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for name, p in procs:
        out = p.communicate()[0].decode(errors="replace")
        # hipcc's host pass does not know the packed-fp32 feature flag; that warning is harmless
        lines = [l for l in out.splitlines() if "packed-fp32-ops" not in l]
        if lines and (verbose or p.returncode):
            print("\n".join(lines), file=sys.stderr)
        if p.returncode:
            failed.append(name)
    if failed:
        raise RuntimeError(what + " failed: " + ", ".join(failed))


def build_library(verbose: bool = False) -> str:
    """The C library: needs hipcc only."""
    cc = hipcc()
    objs = [os.path.join(BUILD, src + ".o") for src in SOURCES]
    run_all("HIP compilation", [(src, [cc] + compile_flags() + ["-c", os.path.join(CSRC, src), "-o", obj])
                                for src, obj in zip(SOURCES, objs)], verbose)
    tmp = LIB_PATH + ".tmp"
    run_all("linking the library", [(LIB_NAME, [cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-soname," + LIB_NAME,
                                                "-o", tmp] + objs)], verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build_binding(verbose: bool = False) -> str:
    """The native half of the Python binding, against the library: needs g++, torch and Python's headers."""
    out = os.path.join(PKG, BINDING_NAME)
    compile_binding, link_binding = binding_commands(os.path.join(BUILD, BINDING + ".o"), out + ".tmp")
    run_all("compiling the Python binding (g++)", [(BINDING, compile_binding)], verbose)
    run_all("linking the Python binding (g++)", [(BINDING_NAME, link_binding)], verbose)
    os.replace(out + ".tmp", out)
    return out


def build(verbose: bool = False) -> str:
    """Always recompiles every source and relinks: the library, then the binding, so that the library is there whole
    where the binding cannot be built."""
    os.makedirs(BUILD, exist_ok=True)
    build_library(verbose)
    build_binding(verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
