"""A launch that fails is reported by the entry point's status and leaves nothing
behind in the CUDA runtime, where the next launch that looks would find it."""
import subprocess

import pytest

from state_space_sequence_chunk_gb300 import build as ssd_build

pytestmark = pytest.mark.gpu
SOURCE = r"""
#include <stdio.h>
#include "ssd_internal.cuh"
__global__ void none(int) {}
int main() {
    // an empty grid, which the host refuses
    const cudaError_t e = ssd::launch_chained(none, dim3(0), dim3(32), 0, nullptr, false, 1);
    const bool left = cudaPeekAtLastError() != cudaSuccess;
    const ssd_status s = ssd::from_cuda(e);
    printf("%d %d %d %d\n", (int)(e != cudaSuccess), (int)left, (int)s, (int)cudaPeekAtLastError());
    return 0;
}
"""


def test_a_failed_launch_leaves_no_error(tmp_path):
    src, exe = str(tmp_path / "launch.cu"), str(tmp_path / "launch")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([ssd_build.nvcc(), *ssd_build.ARCH, *ssd_build.NVCC_FLAGS, "-cudart", "static", "-o", exe, src],
                   check=True, capture_output=True)
    failed, left, status, after = map(int, subprocess.run([exe], check=True, capture_output=True,
                                                          text=True).stdout.split())
    assert (failed, left, status, after) == (1, 1, 7, 0)
