"""AdamW's square root against CUDA's sqrtf, of every fp32 value that is not negative: equal from 2^-80 on, within a unit in the last
place from 2^-126 on, not finite otherwise (zeros, subnormals, infinities, NaNs: the step then calls sqrtf)."""
import ctypes
import os
import subprocess

import pytest
import torch

from ragged_grouped_gemm_device_gb300 import build

pytestmark = pytest.mark.gpu

SOURCE = """
#include "root.cuh"
// of the values with the exponent field blockIdx.y: how many differ, the largest distance in units, how many are finite
__global__ void compare(unsigned* out) {
  unsigned differ = 0, most = 0, finite = 0;
  for (unsigned i = blockIdx.x * blockDim.x + threadIdx.x; i < 1u << 23; i += gridDim.x * blockDim.x) {
    const float v = __uint_as_float(blockIdx.y << 23 | i), a = moe::sqrt_normal(v), b = sqrtf(v);
    const unsigned x = __float_as_uint(a), y = __float_as_uint(b), far = x > y ? x - y : y - x;
    differ += x != y;
    most = far > most ? far : most;
    finite += a * 0.0f == 0.0f;
  }
  atomicAdd(out + 3 * blockIdx.y, differ);
  atomicMax(out + 3 * blockIdx.y + 1, most);
  atomicAdd(out + 3 * blockIdx.y + 2, finite);
}
extern "C" int run(unsigned* out) {
  compare<<<dim3(64, 256), 256>>>(out);
  return cudaGetLastError();
}
"""


def test_every_value(lib, tmp_path):
    src, so = tmp_path / "root_test.cu", tmp_path / "root_test.so"
    src.write_text(SOURCE)
    flags = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC"]
    subprocess.run([build.nvcc(), *build.ARCH, *flags, "-I", build.CSRC, "-shared", str(src), "-o", str(so)], check=True)
    out = torch.zeros(256, 3, dtype=torch.int32, device="cuda")
    call = ctypes.CDLL(os.fspath(so)).run
    call.argtypes = [ctypes.c_void_p]
    torch.cuda.synchronize()
    assert call(out.data_ptr()) == 0
    torch.cuda.synchronize()
    differ, most, finite = out.cpu().T
    assert (finite[1:255] == 1 << 23).all() and finite[0] == 0 and finite[255] == 0
    assert (differ[127 - 80:255] == 0).all() and (most[1:255] <= 1).all()
