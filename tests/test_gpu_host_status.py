"""The host side's error handling, as a program of its own around csrc/host.cuh."""
import os
import subprocess

import pytest

from fine_grained_fp8_sigmoid_b200 import build

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include "host.cuh"
__global__ void nothing() {}
int main() {
  const int failed = moe::cuda_status(cudaSetDevice(1 << 20), "no such device");
  if (failed != MOE_ERR_CUDA) return 1;
  nothing<<<1, 1>>>();
  return moe::launch_status("after it") == MOE_OK ? 0 : 2;
}
"""


def test_a_failed_call_does_not_fail_the_next(lib, tmp_path):
    """A refused runtime call leaves its error in the thread; the launch after it,
    which is fine, must not report it."""
    src, exe = tmp_path / "status.cu", tmp_path / "status"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I", os.path.join(build.HERE, "csrc"), "-o", str(exe), str(src)],
                   check=True)
    assert subprocess.run([str(exe)], timeout=60).returncode == 0
