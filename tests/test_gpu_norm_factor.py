"""The norm's root and reciprocal (csrc/saw_norm.cuh), compiled here as the kernels
compile them, against the correctly rounded built-in ones: every binary32 from
2^-100, the least that a call's eps leaves, to infinity."""
import ctypes
import subprocess

import pytest
import torch

from bit_paged_kv_gb300 import build as saw_build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "saw_norm.cuh"
// how many of the floats [first, first + n) have another root or reciprocal, and the first of them
__global__ void differ(unsigned first, unsigned n, unsigned long long* count, unsigned* least) {
  for (unsigned i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
    const float t = __uint_as_float(first + i), root = __fsqrt_rn(t), r = __frcp_rn(root);
    // (an infinite sum: a factor of 0)
    const float got = saw::norm_root(t);
    if ((t < INFINITY && __float_as_uint(got) != __float_as_uint(root)) ||
        __float_as_uint(saw::norm_factor(t)) != __float_as_uint(r)) {
      atomicAdd(count, 1ull);
      atomicMin(least, first + i);
    }
  }
}
extern "C" int run(unsigned first, unsigned n, void* count, void* least) {
  differ<<<2432, 256>>>(first, n, (unsigned long long*)count, (unsigned*)least);
  return int(cudaDeviceSynchronize());
}
"""


def test_every_float(tmp_path):
    src, lib = tmp_path / "differ.cu", tmp_path / "differ.so"
    src.write_text(SOURCE)
    subprocess.run([saw_build._nvcc(), *saw_build.ARCH, *saw_build.COMMON, "-shared", str(src), "-o", str(lib)], check=True)
    run = ctypes.CDLL(str(lib)).run
    run.argtypes = [ctypes.c_uint, ctypes.c_uint, ctypes.c_void_p, ctypes.c_void_p]
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    least = torch.full((1,), -1, dtype=torch.int32, device="cuda")  # 2^32 - 1
    first, last = (127 - 100) << 23, 0x7F800000         # 2^-100 and infinity
    torch.cuda.synchronize()
    assert run(first, last - first + 1, count.data_ptr(), least.data_ptr()) == 0
    assert count.item() == 0, hex(least.item() & 0xFFFFFFFF)
