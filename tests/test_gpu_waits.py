"""The kernels' bounded waits: a phase that ends late is waited for, one that
never ends is given up after two seconds by the clock, with a status."""
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SOURCE = r"""
#include <cstdio>
#include "ar_tcgen05.cuh"

using namespace ar;

// kind 0: the ring's wait, 1: the attention kernels'.  Thread 32 ends the phase
// after `late` ns (never, if that is 0) and looks at nothing else.
__global__ void wait_kernel(int kind, uint64_t late, uint64_t* out) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int gave_up;
  if (threadIdx.x == 0) {
    mbar_init(smem_addr(&bar), 1);
    gave_up = 0;
  }
  __syncthreads();
  const uint64_t from = global_ns();
  if (threadIdx.x == 32 && late) {
    while (global_ns() < from + late) __nanosleep(1000);
    mbar_arrive(smem_addr(&bar));
  }
  if (threadIdx.x == 0) {
    out[0] = kind ? mbar_wait(smem_addr(&bar), 0, &gave_up) : ring_wait(smem_addr(&bar), 0, &gave_up);
    out[1] = global_ns() - from;
    out[2] = gave_up;
  }
  __syncthreads();
  if (threadIdx.x == 0) out[3] = g_status;
}

int main() {
  uint64_t* out;
  if (cudaMalloc(&out, 32) != cudaSuccess) return 1;
  const uint64_t lates[] = {1000, 20000000, 300000000, 0};
  for (int kind = 0; kind < 2; ++kind)
    for (uint64_t late : lates) {
      uint64_t h[4];
      wait_kernel<<<1, 64>>>(kind, late, out);
      if (cudaMemcpy(h, out, 32, cudaMemcpyDeviceToHost) != cudaSuccess) return 1;
      printf("%d %llu %llu %llu %llu %lld\n", kind, (unsigned long long)late, (unsigned long long)h[0],
             (unsigned long long)h[1], (unsigned long long)h[2], (long long)(int)h[3]);
    }
  return 0;
}
"""


def test_waits(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from allreduce_gradient_reduction_gb300 import binding as ar
    from allreduce_gradient_reduction_gb300 import build as b
    (tmp_path / "waits.cu").write_text(SOURCE)
    at = str(tmp_path / "waits")
    subprocess.run([b.nvcc(), *b.ARCH, "-O2", "-std=c++17", "-I" + b.CSRC, "-o", at, at + ".cu"], check=True,
                   capture_output=True)
    lines = subprocess.run([at], check=True, capture_output=True, text=True, timeout=60, env=dict(os.environ)).stdout
    rows = [[int(x) for x in line.split()] for line in lines.splitlines()]
    assert len(rows) == 8
    for kind, late, came, took, gave_up, status in rows:
        if late:
            assert (came, gave_up) == (1, 0) and late <= took < late + 10 ** 9, (kind, late, took)
        else:
            assert (came, gave_up) == (0, 1) and 1.9e9 < took < 4e9, (kind, took)
            assert kind == 1 or status == ar.AR_ERR_TIMEOUT  # the attention kernels set it where they leave
