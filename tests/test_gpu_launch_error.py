"""A launch that fails is reported by its own call and by no later one. The launch asks for more threads than a block
can have, which the runtime refuses on the host."""
import os
import subprocess

import pytest

from ragged_grouped_gemm_device_gb300 import build

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include "common.cuh"
#include <cstdio>
__global__ void kernel(int) {}
int main() {
  const cudaError_t err = moe::launch_dependent(kernel, 1, 4096, 0, nullptr, 1);
  std::printf("%d %d\n", static_cast<int>(err), static_cast<int>(cudaPeekAtLastError()));
  return 0;
}
"""


def test_a_failed_launch_leaves_no_error_behind(lib, tmp_path):
    src, exe = tmp_path / "launch.cu", tmp_path / "launch"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", build.CSRC, "-I",
                    os.path.join(build.ROOT, "include"), str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out[0] != "0" and out[1] == "0", out
