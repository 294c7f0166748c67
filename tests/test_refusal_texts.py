"""Texts of refusals that name what a call may be given instead (no GPU: a
refused call touches no device)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from test_moe_checks import A, B, BF16, C, D, E, E8M0, F, F32, F4, I32, INVALID, tensor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
SHIM = '#include "gmm_handle.hpp"\nextern "C" void* make() { return new gmm_handle(); }\n'


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """gmm_run on a handle without a device: call -> (status, text)."""
    import moe_grouped_matrix_amd as m
    from moe_grouped_matrix_amd import build
    if not CXX or not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        pytest.skip("no C++ compiler or HIP headers")
    d = tmp_path_factory.mktemp("shim")
    (d / "s.cpp").write_text(SHIM)
    subprocess.run([CXX, "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROCM, "include"),
                    "-I" + os.path.join(ROOT, "include"), "-I" + build.CSRC, str(d / "s.cpp"), "-o", str(d / "s.so")],
                   check=True)
    shim, lib = ctypes.CDLL(str(d / "s.so")), m.load()
    shim.make.restype = ctypes.c_void_p
    h = shim.make()
    raw = ctypes.CDLL(m.LIB_PATH)

    def call(lhs, rhs, rhs_scale, lhs_scale):
        ref = [None if t is None else ctypes.byref(t)
               for t in (lhs, rhs, tensor(C, I32, 2), rhs_scale, None, lhs_scale)]
        got = raw.gmm_run(ctypes.c_void_p(h), *ref, None, 0, ctypes.byref(tensor(F, F32, 8, 16)), None)
        return got, lib.gmm_last_error(h).decode()
    return call


def test_scale_types(run):
    """E8M0 weight scales go with a bf16 lhs and no lhs_scale, too: the text may
    not ask for E8M0 on both sides."""
    lhs, rhs = tensor(A, BF16, 8, 64), tensor(B, F4, 2, 16, 64)
    for scale, lscale in ((tensor(D, BF16, 2, 2, 1, 16), None), (tensor(D, E8M0, 2, 2, 16), None),
                          (tensor(D, F32, 2, 2, 1, 16), tensor(E, E8M0, 8, 2))):
        got, text = run(lhs, rhs, scale, lscale)
        assert got == INVALID
        assert "f32 or E8M0" in text and "rhs_scale" in text and "both sides" not in text
