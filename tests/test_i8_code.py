"""The compiled code of the largest tile of 8-bit products (no GPU): its sums are held in accumulation
registers by the instruction's operands, and the waits between them and what reads them are the
kernel's own, so nothing may come between."""
import os
import re
import shutil
import subprocess

import pytest

from error_bounded_lossy_amd import build


def test_the_sums_of_the_largest_tile_stay_where_they_are():
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not shutil.which(hipcc):
        pytest.skip("no hipcc")
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    out = subprocess.run([hipcc, *flags, "-x", "hip", "--offload-device-only", "-S", os.path.join(build.CSRC, "ec_i8_product.hip"), "-o", "-"],
                         check=True, capture_output=True, text=True).stdout
    kernels = re.findall(r"^(_ZN\S*8i8_tilesILi4ELi4E\S*):\s", out, re.M)
    assert len(kernels) == 12  # three types, dense and by expert, stored as usual and past the caches
    for name in kernels:
        code = out[out.index(f"\n{name}:"):]
        lines = [line.split(";")[0].strip() for line in code[:code.index(".Lfunc_end")].splitlines()]
        lines = [line for line in lines if line and not line.startswith(";")]
        products = [i for i, line in enumerate(lines) if line.startswith("v_mfma")]
        assert len(products) >= 3 * 128, name  # a loop of two stages and a last one
        assert all(re.match(r"v_mfma_i32_16x16x64_i8 a\[(\d+:\d+)\], v\[\S+\], v\[\S+\], a\[\1\]$", lines[i]) for i in products), name
        assert not any("scratch_" in line or "s_swappc" in line for line in lines), name
        first, last = products[0], products[-1]
        assert not any("accvgpr" in line for line in lines[first:last]), name
        # zeros before the barrier in front of the first, and the waits behind the last
        zeros = max(i for i, line in enumerate(lines[:first]) if "v_accvgpr_write" in line)
        assert sum(line.startswith("s_barrier") for line in lines[zeros:first]) >= 1, name
        read = next(i for i in range(last, len(lines)) if "v_accvgpr_read" in lines[i])
        assert lines[last:read].count("s_nop 15") == 2, name
