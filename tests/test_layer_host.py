"""Host arithmetic behind gmm_layer.h, compiled here from the library's own
headers (no GPU): the scale block of a block of 32 elements, found by a
multiplication, and the factors of an AdamW step."""
import ctypes
import math
import os
import random
import subprocess

import numpy as np
import pytest

from test_moe_checks import CXX, ROOT

ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
SOURCE = r"""
#include "gmm_layer_launch.hpp"
extern "C" {
// the first block of 32, below `blocks`, whose scale block is not b / d (-1: none)
long long wrong_block(long long d, long long blocks, long long step) {
  const uint32_t m = gmmk::gmv_magic((int)(32 * d));
  for (long long b = 0; b < blocks; b += step)
    if ((long long)(((unsigned long long)(unsigned)b * m) >> 31) != b / d) return b;
  return -1;
}
void factors(double lr, double b1, double b2, double wd, long long step, float* out) {
  const gmmk::AdamFactors f = gmmk::adam_factors(lr, b1, b2, wd, step);
  out[0] = f.decay; out[1] = f.rate; out[2] = f.root_scale;
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if not CXX or not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        pytest.skip("no C++ compiler or HIP headers")
    d = tmp_path_factory.mktemp("host")
    (d / "c.cpp").write_text(SOURCE)
    subprocess.run([CXX, "-std=c++17", "-O2", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROCM, "include"),
                    "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "moe_grouped_matrix_amd", "csrc"),
                    str(d / "c.cpp"), "-o", str(d / "c.so")], check=True)
    so = ctypes.CDLL(str(d / "c.so"))
    so.wrong_block.restype = ctypes.c_longlong
    so.factors.argtypes = [ctypes.c_double] * 4 + [ctypes.c_longlong, ctypes.c_void_p]
    return so


def test_scale_blocks(lib):
    """Every block of every size up to 256, and the ends of all larger ones, up to K = 2^20."""
    most = 2 ** 15  # blocks of 32 in the largest K
    rng = random.Random(1)
    for d in list(range(1, 257)) + [rng.randint(257, most) for _ in range(300)] + [most - 1, most]:
        assert lib.wrong_block(ctypes.c_longlong(d), ctypes.c_longlong(most), ctypes.c_longlong(1)) == -1, d


def test_factors(lib):
    """Powers by squaring are within some 2 log2(step) roundings of double, far
    below binary32's: each factor is the rounded one, or its neighbour where the
    exact value lies that near to the middle."""
    rng = random.Random(2)
    for step in [1, 2, 3, 7, 100, 1000, 65535, 10 ** 6, 2 ** 31 - 1] + [rng.randint(1, 10 ** 7) for _ in range(200)]:
        lr, b1, b2, wd = rng.random(), rng.choice([0.0, 0.9, 0.99]), rng.choice([0.95, 0.999, 0.9999]), rng.random()
        out = np.zeros(3, np.float32)
        lib.factors(lr, b1, b2, wd, step, out.ctypes.data)
        want = (1 - lr * wd, lr / (1 - b1 ** step), 1 / math.sqrt(1 - b2 ** step))
        for got, w in zip(out, want):
            assert abs(float(got) - w) <= abs(w) * 2.0 ** -24 * 1.0001, (step, got, w)
