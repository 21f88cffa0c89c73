"""The waits of the attention kernels give up after the documented 2 s of device
time.  A kernel of one warp, built here from the library's own header, waits on a
barrier that nothing completes; it returns by itself and reports how long it took."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

SOURCE = r"""
#include "attn_common.cuh"
using namespace tqi;

__global__ void wait_kernel(int which, unsigned long long* out) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    sm100::mbar_init(&bar, 1);
    sm100::fence_mbar_init();
  }
  __syncthreads();
  // parity 1: the phase before the first, complete from the start; parity 0: nothing completes it
  const bool at_once = attn::wait_warp(&bar, 1);
  const uint64_t t0 = sm100::globaltimer();
  const bool ok = which ? sm100::mbar_wait_warp(&bar, 0) : attn::wait_warp(&bar, 0);
  const uint64_t t1 = sm100::globaltimer();
  if (threadIdx.x == 0) out[0] = t1 - t0, out[1] = ok, out[2] = at_once;
}

extern "C" int run(int which, unsigned long long* host) {
  unsigned long long* dev = nullptr;
  cudaError_t e = cudaMalloc(&dev, 24);
  if (e == cudaSuccess) wait_kernel<<<1, 32>>>(which, dev);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpy(host, dev, 24, cudaMemcpyDeviceToHost);
  cudaFree(dev);
  return (int)e;
}
"""


def test_a_wait_that_nothing_ends_gives_up_after_two_seconds(root, tmp_path):
    src, lib = tmp_path / "wait.cu", tmp_path / "wait.so"
    src.write_text(SOURCE)
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or shutil.which("/usr/local/cuda/bin/nvcc")
    if not nvcc:
        pytest.skip("needs nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O3", "-shared", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(root, "compressed_kv_cache_turboquant_b200", "csrc"), "-I", os.path.join(root, "include"),
                    str(src), "-o", str(lib)], check=True)
    torch.cuda.synchronize()
    fn = ctypes.CDLL(str(lib)).run
    for which in (0, 1):
        got = (ctypes.c_ulonglong * 3)()
        assert fn(which, got) == 0
        ns, completed, at_once = got
        assert at_once and not completed
        # a try before the clock is read (200 us at most), one behind the limit, and the timer's steps
        assert 2.0e9 <= ns <= 2.05e9, ns / 1e9
