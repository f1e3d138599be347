"""The compiled code of the norm (no GPU): its rows and sums stay in registers."""
import os
import re
import shutil
import subprocess

import pytest

from error_bounded_lossy_amd import build


def test_no_kernel_keeps_its_rows_in_memory():
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not shutil.which(hipcc):
        pytest.skip("no hipcc")
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    out = subprocess.run([hipcc, *flags, "-x", "hip", "--offload-device-only", "-S", os.path.join(build.CSRC, "ec_norm.hip"), "-o", "-"],
                         check=True, capture_output=True, text=True).stdout
    kernels = re.findall(r"^(_ZN\S*(?:rms_norm|column_sums)\S*):\s", out, re.M)
    assert len(kernels) == 40  # 24 of the norm, 12 of its gradients, 4 of column sums
    for name in kernels:
        code = out[out.index(f"\n{name}:"):]
        code = code[:code.index(".Lfunc_end")]
        assert "s_endpgm" in code and "scratch_" not in code and "s_swappc" not in code, name
