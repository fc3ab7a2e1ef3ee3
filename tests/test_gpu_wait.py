"""A wait of the dense attention kernel that runs out: nothing ever arrives on
its barrier.  It returns within seconds and says so, and the waits behind it
return at once; the kernel ends by itself."""
import subprocess

import pytest

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <cstdio>
#include <cuda_runtime.h>
#include "kv_tc.cuh"
__global__ void waits(long long *clocks, unsigned *dead_after) {
  __shared__ unsigned long long bars[3];
  __shared__ unsigned dead;
  if (threadIdx.x == 0) {
    for (auto &b : bars) kv::bar_init(kv::s32(&b), 1);
    dead = 0;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  const int order[3] = {0, 1, 2};  // arrived, never arrived, never arrived
  kv::bar_arrive(kv::s32(&bars[0]));
  for (int i : order) {
    const long long t = clock64();
    kv::bar_wait(kv::s32(&bars[i]), 0, &dead);
    clocks[i] = clock64() - t;
    dead_after[i] = dead;
  }
}
int main() {
  long long *c;
  unsigned *d;
  if (cudaMallocManaged(&c, 24) || cudaMallocManaged(&d, 12)) return 1;
  waits<<<1, 32>>>(c, d);
  if (cudaGetLastError() || cudaDeviceSynchronize()) return 2;
  printf("%lld %lld %lld %u %u %u\n", c[0], c[1], c[2], d[0], d[1], d[2]);
  return 0;
}
"""


def test_a_wait_gives_up(tmp_path):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verify_03_gb300 as sv
    (tmp_path / "wait.cu").write_text(SOURCE)
    exe = str(tmp_path / "wait")
    subprocess.run(["nvcc", *[f for f in sv._NVCC_FLAGS if f not in ("-Xcompiler", "-fPIC")],
                    str(tmp_path / "wait.cu"), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=120).stdout.split()
    clocks, dead = [int(x) for x in out[:3]], [int(x) for x in out[3:]]
    assert dead == [0, 1, 1]
    assert clocks[0] < 10 ** 5 and clocks[2] < 10 ** 5
    assert 10 ** 8 < clocks[1] < 2 * 10 ** 10  # a tenth of a second to ten, at 1 to 2 GHz
