"""Builds libtq2.so in-tree with hipcc for gfx950, and the Python calls' module beside it.

Flags: -O3, C++17, position-independent shared object; packed-FP32 VALU ops are
disabled for the device code (-Xclang -target-feature -Xclang -packed-fp32-ops).
Each source is compiled to an object of its own, several at a time.  The module
(csrc/binding.cpp) is host code against Python's and torch's headers.
"""

from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtq2.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["moe_few.hip", "q4_linear.hip", "block_norm.hip", "q4_tiled.hip", "q4_gemm.hip", "q4_group.hip", "q4_moe.hip",
           "moe_route.hip", "moe_layer.hip", "libtq2.cpp", "libq4.cpp", "libblock.cpp", "repack.cpp", "tq2_gemv.hip", "mfma_gemm.hip", "blr.hip", "skinny_gemm.hip"]
ARCH = "gfx950"


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "hipcc"


def compile_cmd(source: str, out: str, extra=()) -> list:
    return [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-c",
            "-x", "hip", os.path.join(CSRC, source),
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-result", *extra, "-o", out]


def binding_cmd(out: str) -> list:
    import torch

    t = os.path.dirname(torch.__file__)
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(a for d in (f"{t}/include", f"{t}/include/torch/csrc/api/include", "/opt/rocm/include",
                          sysconfig.get_paths()["include"]) for a in ("-isystem", d)),
            os.path.join(CSRC, "binding.cpp"), "-o", out, f"-L{t}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_hip"]


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory(prefix="tq2_build_") as d:
        objs = [os.path.join(d, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        cmds = [compile_cmd(s, o) for s, o in zip(SOURCES, objs)] + [binding_cmd(BINDING + ".tmp")]
        if verbose:
            print("\n".join(" ".join(c) for c in cmds), flush=True)
        with ThreadPoolExecutor(min(6, os.cpu_count() or 1)) as pool:
            for r in [pool.submit(subprocess.run, c, check=True) for c in cmds]:
                r.result()
        subprocess.run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp], check=True)
    os.replace(BINDING + ".tmp", BINDING)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
    sys.exit(0)
