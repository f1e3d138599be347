"""Build the HIP library libec.so (gfx950) in-tree with hipcc.

Flags: IEEE fp32 everywhere (-ffp-contract=off, no fast-math, correctly
rounded division is hipcc's default), packed-fp32 instructions disabled.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libec.so")
SOURCES = [os.path.join(CSRC, name) for name in
           ("ec_kernels.hip", "ec_huffman.hip", "ec_mx.hip", "ec_mx_product.hip", "ec_i8.hip",
            "ec_i8_product.hip", "ec_norm.hip", "ec_route.hip", "ec_experts.hip",
            "ec_runtime.cpp")]
ARCH = os.environ.get("EC_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    f"-I{os.path.join(ROOT, 'include')}",
]


def build(verbose: bool = False) -> str:
    """Every source is compiled, several at a time, and the objects linked."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    jobs = int(os.environ.get("MAX_JOBS") or min(8, os.cpu_count() or 1))
    with tempfile.TemporaryDirectory() as objects:
        def compile(source: str) -> str:
            out = os.path.join(objects, os.path.basename(source) + ".o")
            cmd = [hipcc, *HIPCC_FLAGS, "-c", "-x", "hip", source, "-o", out]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True, cwd=CSRC)
            return out

        with ThreadPoolExecutor(max(1, jobs)) as pool:
            made = list(pool.map(compile, SOURCES))
        tmp = LIB + ".tmp"
        subprocess.run([hipcc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *made, "-o", tmp],
                       check=True, cwd=CSRC)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    print(LIB)
    sys.exit(0)
