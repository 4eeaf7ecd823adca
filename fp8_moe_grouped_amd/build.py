"""Build libfp8_moe_grouped.so in-tree with hipcc for gfx950, and the binding's
extension with the host compiler.

Each HIP source is compiled to an object under ``_build/`` (in parallel) and
linked into ``fp8_moe_grouped_amd/libfp8_moe_grouped.so``; ``csrc/calls.cpp``,
host code against torch's headers, becomes ``fp8_moe_grouped_amd/_calls.so``.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfp8_moe_grouped.so")
CALLS = os.path.join(PKG, "_calls.so")

SOURCES = ["quant.hip", "gmm_fwd.hip", "dlhs.hip", "tgmm.hip", "dequant.hip", "route.hip", "permute.hip", "mxfp4.hip",
           "gmm_mxfp4.hip", "api.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # keep the compiler from forming packed-f32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in p.stdout.splitlines() if "packed-fp32-ops" not in l)
    if p.returncode != 0:
        raise RuntimeError(f"command failed ({p.returncode}): {' '.join(cmd)}\n{out}")
    return out


def build_calls() -> str:
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{p}" for p in (*include_paths("cuda"), sysconfig.get_path("include"))),
           os.path.join(CSRC, "calls.cpp"), "-o", CALLS + ".tmp", *(f"-L{p}" for p in library_paths("cuda")),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    log = _run(cmd)
    os.replace(CALLS + ".tmp", CALLS)
    return log


def build(verbose: bool = False, jobs: int | None = None) -> str:
    """Compile every source and link the shared library and the extension; returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    objs = [os.path.join(BUILD, os.path.splitext(s)[0] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        return _run([HIPCC, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj])

    jobs = jobs or min(8, os.cpu_count() or 4)
    with ThreadPoolExecutor(jobs) as ex:
        calls = ex.submit(build_calls)
        logs = list(ex.map(compile_one, zip(srcs, objs)))
        tmp = LIB + ".tmp"
        logs.append(_run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]))
        os.replace(tmp, LIB)
        logs.append(calls.result())     # last: the library stands without the extension, whose failure is raised here
    if verbose:
        for l in logs:
            if l.strip():
                print(l)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
