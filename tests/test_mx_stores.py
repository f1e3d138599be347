"""Stores past the caches are in the code that the compiler makes: where the two branches of a store
ended alike, it made one store of them, without the hint.  A kernel of the same shape is compiled
(no GPU) with the library's flags."""
import os
import shutil
import subprocess

import pytest

from error_bounded_lossy_amd import build

KERNELS = """
#include "ec_mx_device.h"
using namespace ecmx;
template <typename T> __device__ void body(const uint32_t* v, T* y, uint32_t n, bool past) {
  uint32_t w[4];
  __builtin_memcpy(w, v + threadIdx.x * 4, 16);
  T* to = y + threadIdx.x * (16 / sizeof(T));
  if (threadIdx.x < n) store16(to, w, past);
}
template <typename T> __device__ void rows(const T* x, T* y, int64_t n, bool past) {
  store_eight(y + threadIdx.x * 8, n, load_eight(x + threadIdx.x * 8, 8), past);
}
extern "C" __global__ void values_bf16(const uint32_t* v, bf16_t* y, uint32_t n, bool past) { body(v, y, n, past); }
extern "C" __global__ void values_fp16(const uint32_t* v, f16_t* y, uint32_t n, bool past) { body(v, y, n, past); }
extern "C" __global__ void values_fp32(const uint32_t* v, float* y, uint32_t n, bool past) { body(v, y, n, past); }
extern "C" __global__ void rows_bf16(const bf16_t* x, bf16_t* y, int64_t n, bool past) { rows(x, y, n, past); }
"""


def test_the_hint_survives_the_compiler(tmp_path):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not shutil.which(hipcc):
        pytest.skip("no hipcc")
    source = tmp_path / "stores.hip"
    source.write_text(KERNELS)
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    out = subprocess.run([hipcc, *flags, f"-I{build.CSRC}", "-x", "hip", "--offload-device-only", "-S", str(source), "-o", "-"],
                         check=True, capture_output=True, text=True).stdout
    for name in ("values_bf16", "values_fp16", "values_fp32", "rows_bf16"):
        code = out[out.index(f"\n{name}:"):]
        code = code[:code.index("s_endpgm")]
        stores = [line for line in code.splitlines() if "global_store_dwordx4" in line]
        past = [line for line in stores if line.split(";")[0].rstrip().endswith(" nt")]
        assert past and len(past) < len(stores), (name, stores)
