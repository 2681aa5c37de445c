"""Bounded waits of the low-bit kernels: a thread whose wait ran out still takes part in what its warp and its fellow
warps do together, so that the kernel ends with an error status instead of standing at a barrier."""
import ctypes
import os
import subprocess

import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from long_context_compressed_hca_b200 import build as hbuild

KERNEL = """
#include "lowbit.cuh"
// Four warps, each waiting at a barrier of its own; nothing arrives at the second's.  All meet at a named barrier
// after the first wait and after a second one.
__global__ void waits(int *status, int *out, long long *cycles) {
  __shared__ uint64_t bars[4];
  __shared__ uint32_t ran_out;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) hca::mbar_init(hca::smem_u32(&bars[i]), 1);
    ran_out = 0u;
    hca::mbar_fence_init();
  }
  __syncthreads();
  if (lane == 0 && warp != 1) hca::mbar_arrive(hca::smem_u32(&bars[warp]));
  const long long t0 = clock64();
  const hca::Waits wait{status, &ran_out};
  for (int i = 0; i < 2; ++i) {
    wait(hca::smem_u32(&bars[warp]), 0);
    asm volatile("bar.sync 1, 128;" ::: "memory");
  }
  out[threadIdx.x] = wait.out;
  if (threadIdx.x == 0) *cycles = clock64() - t0;
}
extern "C" int run_waits(int *status, int *out, long long *cycles) {
  waits<<<1, 128>>>(status, out, cycles);
  return (int)cudaDeviceSynchronize();
}
"""


@pytest.mark.gpu
def test_warps_meet_after_a_wait_that_ran_out(cuda, tmp_path):
    src, so = tmp_path / "waits.cu", tmp_path / "waits.so"
    src.write_text(KERNEL)
    subprocess.run([hbuild.nvcc(), "-shared", str(src), "-o", str(so), *hbuild.ARCH, *hbuild.FLAGS], check=True,
                   capture_output=True)
    status, out = torch.zeros(1, dtype=torch.int32, device=cuda), torch.full((128,), -1, dtype=torch.int32, device=cuda)
    cycles = torch.zeros(1, dtype=torch.int64, device=cuda)
    torch.cuda.synchronize()
    f = ctypes.CDLL(str(so)).run_waits
    f.argtypes = [ctypes.c_void_p] * 3
    assert f(status.data_ptr(), out.data_ptr(), cycles.data_ptr()) == 0
    assert status.item() == hb.HCA_ERR_TIMEOUT
    assert out.view(4, 32).tolist() == [[0] * 32, [1] * 32, [0] * 32, [0] * 32]
    assert 4e9 <= cycles.item() < 8e9          # one limit, not one per wait


def test_only_lanes_on_their_own_leave_on_a_wait():
    """Named barriers, votes and shuffles need every lane and warp of a role: leaving a role on a wait is for the loads
    that one lane issues by itself."""
    leaving = []
    for name in ("attend_fp4.cu", "w4.cu"):
        with open(os.path.join(hbuild.CSRC, name)) as f:
            leaving += [x.strip() for x in f if "wait" in x and ("break;" in x or "return;" in x or "return false;" in x)]
    assert len(leaving) == 2 and all("c_empty" in x or "x_empty" in x for x in leaving), leaving
