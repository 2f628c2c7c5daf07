"""Build libmoe.so in-tree with nvcc for sm_103a (GB300).

Each CUDA translation unit compiles in parallel to an object file; the objects
link into ``expert_routed_ffn_gb300/_build/libmoe.so`` (CUDA runtime linked
statically, the driver's tensor-map encoder fetched at run time).  A unit is
recompiled when it, or a header, is newer than its object.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmoe.so")

SOURCES = ["router.cu", "router_tc.cu", "stream.cu", "gemm_tc.cu", "gemm_sab.cu", "gemm_mxt.cu", "moe_capi.cu",
           "dispatch_static.cu", "op_capi.cu", "grouped.cu", "mx_quant.cu", "mx_grouped.cu",
           "grad_clip.cu", "gated.cu", "norm.cu", "orthogonalize.cu"]
HEADERS = [os.path.join(CSRC, "common.cuh"), os.path.join(CSRC, "kernels.h"), os.path.join(CSRC, "routing.cuh"),
           os.path.join(CSRC, "op_host.h"), os.path.join(CSRC, "grouped.cuh"), os.path.join(CSRC, "gated.cuh"),
           os.path.join(CSRC, "grouped_kernel.cuh"), os.path.join(INCLUDE, "moe.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, extra_flags=(), out_dir: str = BUILD) -> str:
    """Compile into out_dir (default: the package's _build) and link libmoe.so there."""
    os.makedirs(out_dir, exist_ok=True)
    lib = os.path.join(out_dir, "libmoe.so")
    nvcc = _nvcc()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(out_dir, src.replace(".cu", ".o"))
        objs.append(o)
        if _stale(o, [s] + HEADERS):
            jobs.append([nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        for msg in ex.map(run, jobs):
            if verbose and msg:
                print(msg, file=sys.stderr)
    if jobs or _stale(lib, objs):
        tmp = lib + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
