"""Builds libtq2.so in-tree with hipcc for gfx950.

Flags: -O3, C++17, position-independent shared object; packed-FP32 VALU ops are
disabled for the device code (-Xclang -target-feature -Xclang -packed-fp32-ops).
Each source is compiled to an object of its own, several at a time.
"""

from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtq2.so")
SOURCES = ["q4_tiled.hip", "q4_gemm.hip", "q4_group.hip", "q4_moe.hip", "moe_route.hip", "libtq2.cpp", "libq4.cpp", "repack.cpp", "tq2_gemv.hip",
           "mfma_gemm.hip", "blr.hip", "skinny_gemm.hip"]
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


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory(prefix="tq2_build_") as d:
        objs = [os.path.join(d, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        cmds = [compile_cmd(s, o) for s, o in zip(SOURCES, objs)]
        if verbose:
            print("\n".join(" ".join(c) for c in cmds), flush=True)
        with ThreadPoolExecutor(min(6, os.cpu_count() or 1)) as pool:
            for r in [pool.submit(subprocess.run, c, check=True) for c in cmds]:
                r.result()
        subprocess.run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
    sys.exit(0)
