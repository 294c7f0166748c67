"""Refusals of the entry points of include/gmm_moe.h on the CPU: the argument
checks are plain host C++, compiled here with the C++ compiler and called
through ctypes (no GPU, no library)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")

F32, BF16, E4M3, I32, E5M2, E8M0, I8, I4, U4, F4, I64 = range(11)
OK, INVALID, UNSUPPORTED = 0, -1, -2

SOURCE = r"""
#include "gmm_moe_checks.hpp"
using namespace gmmh;
typedef const gmm_tensor* T;
static thread_local std::string text;
static int say(const Check& c) { text = c.text; return c.status; }
extern "C" {
const char* why() { return text.c_str(); }
int sort_tokens(T a, T b, T c, const void* w, size_t n) { return say(check_sort_tokens(a, b, c, w, n)); }
int dispatch(T a, T b, T c) { return say(check_dispatch(a, b, c)); }
int combine(T a, T b, T c, T d) { return say(check_combine(a, b, c, d)); }
int combine_grad(T a, T b, T c, T d, T e, T f) { return say(check_combine_grad(a, b, c, d, e, f)); }
int quant(T a, T b, T c) { return say(check_mxfp4(a, b, c, true)); }
int widen(T a, T b, T c) { return say(check_mxfp4(c, a, b, false)); }
void split(long long n, long long g, long long* out) {
  const SortSplit s = sort_split(n, g);
  out[0] = s.blocks; out[1] = s.per; out[2] = (long long)sort_workspace_bytes(n, g);
}
}
"""


class Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if not CXX:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("checks")
    (d / "c.cpp").write_text(SOURCE)
    subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared",
                    "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "moe_grouped_matrix_amd", "csrc"),
                    str(d / "c.cpp"), "-o", str(d / "c.so")], check=True)
    so = ctypes.CDLL(str(d / "c.so"))
    so.why.restype = ctypes.c_char_p
    return so


def tensor(at, dtype, *shape):
    return Tensor(at, dtype, len(shape), (ctypes.c_int64 * 4)(*shape))


# device addresses far apart: 1 TiB each
A, B, C, D, E, F = ((i + 1) << 40 for i in range(6))


def call(lib, name, *args):
    fn = getattr(lib, name)
    got = fn(*[ctypes.byref(a) if isinstance(a, Tensor) else a for a in args])
    return got, lib.why().decode()


def refused(lib, status, word, name, *args):
    got, text = call(lib, name, *args)
    assert got == status, (name, got, text)
    assert word in text, text


def good(lib, name, *args):
    got, text = call(lib, name, *args)
    assert got == OK, (name, text)


def sort_args(ids=I64, T=5, k=8, G=16, ws=None, n=0):
    return [tensor(A, ids, T, k), tensor(B, I32, G), tensor(C, I32, T, k), ctypes.c_void_p(ws), ctypes.c_size_t(n)]


def test_sort_accepts(lib):
    good(lib, "sort_tokens", *sort_args())
    good(lib, "sort_tokens", *sort_args(I32, 0, 1, 1))
    good(lib, "sort_tokens", *sort_args(I32, 1, 64, 1024))
    out = (ctypes.c_longlong * 3)()
    lib.split(ctypes.c_longlong(32768 * 8), ctypes.c_longlong(128), out)
    good(lib, "sort_tokens", *sort_args(I64, 32768, 8, 128, D, out[2]))


def test_sort_refuses(lib):
    a = sort_args()
    refused(lib, INVALID, "required", "sort_tokens", None, *a[1:])
    refused(lib, INVALID, "int32 or int64", "sort_tokens", tensor(A, F32, 5, 8), *a[1:])
    refused(lib, INVALID, "(T, k)", "sort_tokens", tensor(A, I64, 40), *a[1:])
    refused(lib, INVALID, "k >= 1", "sort_tokens", tensor(A, I64, 5, 0), *a[1:])
    refused(lib, UNSUPPORTED, "64 choices", "sort_tokens", tensor(A, I64, 5, 65), *a[1:])
    refused(lib, UNSUPPORTED, "2^31", "sort_tokens", tensor(A, I64, 1 << 28, 8), *a[1:])
    refused(lib, UNSUPPORTED, "2^31", "sort_tokens", tensor(A, I64, 1 << 62, 64), *a[1:])
    refused(lib, INVALID, "group_sizes", "sort_tokens", a[0], tensor(B, I64, 16), *a[2:])
    refused(lib, INVALID, "one group", "sort_tokens", a[0], tensor(B, I32, 0), *a[2:])
    refused(lib, UNSUPPORTED, "1024 groups", "sort_tokens", a[0], tensor(B, I32, 1025), *a[2:])
    refused(lib, INVALID, "slot_row", "sort_tokens", a[0], a[1], tensor(C, I32, 8, 5), *a[3:])
    refused(lib, INVALID, "slot_row", "sort_tokens", a[0], a[1], tensor(C, I64, 5, 8), *a[3:])
    refused(lib, INVALID, "null", "sort_tokens", tensor(None, I64, 5, 8), *a[1:])
    refused(lib, INVALID, "16-byte", "sort_tokens", tensor(A + 8, I64, 5, 8), *a[1:])
    refused(lib, INVALID, "overlaps an input", "sort_tokens", a[0], a[1], tensor(A + 16, I32, 5, 8), *a[3:])
    refused(lib, INVALID, "two outputs", "sort_tokens", a[0], a[1], tensor(B, I32, 5, 8), *a[3:])


def test_sort_workspace(lib):
    big = sort_args(I64, 32768, 8, 128, D, 8)
    refused(lib, INVALID, "workspace needs", "sort_tokens", *big)
    refused(lib, INVALID, "workspace needs", "sort_tokens", *big[:3], ctypes.c_void_p(None), ctypes.c_size_t(1 << 20))
    refused(lib, INVALID, "16-byte", "sort_tokens", *big[:3], ctypes.c_void_p(D + 4), ctypes.c_size_t(1 << 20))
    refused(lib, INVALID, "workspace overlaps", "sort_tokens", *big[:3], ctypes.c_void_p(C), ctypes.c_size_t(1 << 20))
    out = (ctypes.c_longlong * 3)()
    for n in (0, 1, 4095, 4096, 4097, 5000, 262144, 262145, 1 << 24, (1 << 31) - 1):
        for g in (1, 2, 128, 1000, 1024):
            lib.split(ctypes.c_longlong(n), ctypes.c_longlong(g), out)
            blocks, per, ws = out
            assert blocks >= 1 and blocks * per >= n and (blocks - 1) * per < max(n, 1), (n, g, blocks, per)
            if blocks == 1:
                assert ws == 0 and n <= 4096
            else:
                assert ws == blocks * (g + 1) * 4 and per % 1024 == 0 and blocks <= 256


def test_dispatch(lib):
    s = tensor(B, I32, 5, 8)
    for dt in (F32, BF16, E4M3, E5M2, E8M0, I8, I32):
        good(lib, "dispatch", tensor(A, dt, 5, 33), s, tensor(C, dt, 40, 33))
    good(lib, "dispatch", tensor(None, BF16, 0, 33), tensor(None, I32, 0, 8), tensor(None, BF16, 0, 33))
    x, o = tensor(A, BF16, 5, 33), tensor(C, BF16, 40, 33)
    refused(lib, INVALID, "required", "dispatch", x, None, o)
    refused(lib, INVALID, "int32", "dispatch", x, tensor(B, I64, 5, 8), o)
    refused(lib, INVALID, "dtype", "dispatch", tensor(A, F4, 5, 32), s, tensor(C, F4, 40, 32))
    refused(lib, INVALID, "2-tensor", "dispatch", tensor(A, BF16, 5, 3, 11), s, o)
    refused(lib, INVALID, "expected x", "dispatch", tensor(A, BF16, 6, 33), s, o)
    refused(lib, INVALID, "expected out", "dispatch", x, s, tensor(C, BF16, 39, 33))
    refused(lib, INVALID, "dtype", "dispatch", x, s, tensor(C, F32, 40, 33))
    refused(lib, INVALID, "extent", "dispatch", tensor(A, BF16, 5, 0), s, tensor(C, BF16, 40, 0))
    refused(lib, UNSUPPORTED, "2^28", "dispatch", tensor(A, BF16, 5, 1 << 28), s, tensor(C, BF16, 40, 1 << 28))
    refused(lib, INVALID, "overlaps an input", "dispatch", x, s, tensor(A, BF16, 40, 33))
    refused(lib, INVALID, "16-byte", "dispatch", tensor(A + 2, BF16, 5, 33), s, o)


def test_combine(lib):
    s = tensor(B, I32, 5, 8)
    r, w, o = tensor(A, BF16, 40, 33), tensor(C, F32, 5, 8), tensor(D, F32, 5, 33)
    good(lib, "combine", r, s, w, o)
    good(lib, "combine", r, s, None, tensor(D, BF16, 5, 33))
    good(lib, "combine", tensor(A, F32, 40, 33), s, tensor(C, BF16, 5, 8), o)
    refused(lib, INVALID, "required", "combine", None, s, w, o)
    refused(lib, INVALID, "f32 or bf16", "combine", tensor(A, E4M3, 40, 33), s, w, o)
    refused(lib, INVALID, "f32 or bf16", "combine", r, s, w, tensor(D, I32, 5, 33))
    refused(lib, INVALID, "weights", "combine", r, s, tensor(C, I32, 5, 8), o)
    refused(lib, INVALID, "weights", "combine", r, s, tensor(C, F32, 40), o)
    refused(lib, INVALID, "expected rows", "combine", tensor(A, BF16, 41, 33), s, w, o)
    refused(lib, INVALID, "expected out", "combine", r, s, w, tensor(D, F32, 5, 34))
    refused(lib, INVALID, "overlaps an input", "combine", r, s, w, tensor(A + 64, F32, 5, 33))


def test_combine_grad(lib):
    s = tensor(B, I32, 5, 8)
    g, r, w = tensor(A, F32, 5, 33), tensor(C, BF16, 40, 33), tensor(D, F32, 5, 8)
    dr, dw = tensor(E, BF16, 40, 33), tensor(F, F32, 5, 8)
    good(lib, "combine_grad", g, r, s, w, dr, dw)
    refused(lib, INVALID, "required", "combine_grad", g, r, s, None, dr, dw)
    refused(lib, INVALID, "drows", "combine_grad", g, r, s, w, tensor(E, F32, 40, 33), dw)
    refused(lib, INVALID, "dweights", "combine_grad", g, r, s, w, dr, tensor(F, BF16, 5, 8))
    refused(lib, INVALID, "dweights", "combine_grad", g, r, s, w, dr, tensor(F, F32, 8, 5))
    refused(lib, INVALID, "expected dout", "combine_grad", tensor(A, F32, 4, 33), r, s, w, dr, dw)
    refused(lib, INVALID, "overlaps an input", "combine_grad", g, r, s, w, tensor(C, BF16, 40, 33), dw)
    refused(lib, INVALID, "two outputs", "combine_grad", g, r, s, w, dr, tensor(E + 32, F32, 5, 8))


def test_mxfp4(lib):
    good(lib, "quant", tensor(A, BF16, 7, 96), tensor(B, F4, 7, 96), tensor(C, E8M0, 7, 3))
    good(lib, "quant", tensor(A, F32, 2, 7, 96), tensor(B, F4, 2, 7, 96), tensor(C, E8M0, 2, 3, 1, 7))
    good(lib, "widen", tensor(B, F4, 7, 96), tensor(C, E8M0, 7, 3), tensor(A, F32, 7, 96))
    good(lib, "quant", tensor(None, BF16, 0, 96), tensor(None, F4, 0, 96), tensor(None, E8M0, 0, 3))
    x, q, s = tensor(A, BF16, 7, 96), tensor(B, F4, 7, 96), tensor(C, E8M0, 7, 3)
    for name in ("quant", "widen"):
        def args(x=x, q=q, s=s):
            return (x, q, s) if name == "quant" else (q, s, x)
        refused(lib, INVALID, "required", name, *args(q=None))
        refused(lib, INVALID, "f32 or bf16", name, *args(x=tensor(A, E4M3, 7, 96)))
        refused(lib, INVALID, "2- or 3-tensor", name, *args(x=tensor(A, BF16, 96)))
        refused(lib, INVALID, "32-element", name, *args(x=tensor(A, BF16, 7, 48), q=tensor(B, F4, 7, 48)))
        refused(lib, INVALID, "q must", name, *args(q=tensor(B, I8, 7, 96)))
        refused(lib, INVALID, "q must", name, *args(q=tensor(B, F4, 7, 48)))
        refused(lib, INVALID, "scale must", name, *args(s=tensor(C, E8M0, 3, 7)))
        refused(lib, INVALID, "scale must", name, *args(s=tensor(C, F32, 7, 3)))
        refused(lib, INVALID, "extent", name, *args(x=tensor(A, BF16, -7, 96)))
        refused(lib, UNSUPPORTED, "2^31 rows", name, *args(x=tensor(A, BF16, 1 << 31, 96)))
        refused(lib, UNSUPPORTED, "2^28", name, *args(x=tensor(A, BF16, 7, 1 << 28)))
        refused(lib, INVALID, "16-byte", name, *args(q=tensor(B + 8, F4, 7, 96)))
        refused(lib, INVALID, "overlap", name, *args(q=tensor(A, F4, 7, 96)))
    refused(lib, INVALID, "scale must", "quant", tensor(A, F32, 2, 7, 96), tensor(B, F4, 2, 7, 96),
            tensor(C, E8M0, 2, 7, 3))
    refused(lib, INVALID, "two outputs", "quant", x, q, tensor(B + 16, E8M0, 7, 3))


def test_header_and_binding_agree():
    """gmm_moe.h's entry points are the binding's, the library exports them
    and the flag bit is the same."""
    import moe_grouped_matrix_amd as m
    from moe_grouped_matrix_amd import _moe, build
    text = open(os.path.join(ROOT, "include", "gmm_moe.h")).read()
    flags = re.findall(r"#define (GMM_FLAG_\w+) (0x[0-9a-fA-F]+)u", text)
    assert [(k, int(v, 16)) for k, v in flags] == [("GMM_FLAG_BAD_ROW", m.FLAG_BAD_ROW)]
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = sorted(set(re.findall(r"^\s*gmm_status\s+(gmm_\w+)\s*\(", code, flags=re.M)))
    assert declared == sorted(m.EXPORTED_MOE)
    if not os.path.exists(m.LIB_PATH):
        build.build()
    lib = m.load()
    for name in declared:
        assert hasattr(lib, name) and getattr(lib, name).argtypes, name
    assert _moe.GMM_I64 == I64


def test_workspace_query_refuses():
    import moe_grouped_matrix_amd as m
    lib = m.load()
    n = ctypes.c_size_t(7)
    assert lib.gmm_sort_tokens_workspace(262144, 128, ctypes.byref(n)) == OK and n.value > 0
    assert lib.gmm_sort_tokens_workspace(8, 128, ctypes.byref(n)) == OK and n.value == 0
    assert lib.gmm_sort_tokens_workspace(-1, 128, ctypes.byref(n)) == INVALID and n.value == 0
    assert lib.gmm_sort_tokens_workspace(8, 0, ctypes.byref(n)) == INVALID
    assert lib.gmm_sort_tokens_workspace(8, 1025, ctypes.byref(n)) == UNSUPPORTED
    assert lib.gmm_sort_tokens_workspace(1 << 31, 8, ctypes.byref(n)) == UNSUPPORTED
    assert lib.gmm_sort_tokens_workspace(8, 8, None) == INVALID


def test_null_handle_is_refused():
    import moe_grouped_matrix_amd as m
    lib = m.load()
    assert lib.gmm_sort_tokens_run(None, None, None, None, None, 0, None) == INVALID
    assert lib.gmm_dispatch_run(None, None, None, None, None) == INVALID
    assert lib.gmm_combine_run(None, None, None, None, None, None) == INVALID
    assert lib.gmm_combine_grad_run(None, None, None, None, None, None, None, None) == INVALID
    assert lib.gmm_quant_mxfp4_run(None, None, None, None, None) == INVALID
    assert lib.gmm_widen_mxfp4_run(None, None, None, None, None) == INVALID


def test_binding_refuses_host_tensors():
    import torch

    import moe_grouped_matrix_amd as m
    ids, x = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 64, dtype=torch.bfloat16)
    slots, rows = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, 64)
    for call_ in (lambda: m.sort_tokens(ids, 4), lambda: m.dispatch(x, slots), lambda: m.combine(rows, slots),
                  lambda: m.combine_grad(x, rows, slots, torch.zeros(4, 2)), lambda: m.quant_mxfp4(x),
                  lambda: m.widen_mxfp4(x.to(torch.uint8), x)):
        with pytest.raises(m.GmmInvalid, match="device tensor"):
            call_()


def test_the_compiled_binding_leaves_what_it_does_not_take():
    """Without a device every call comes back as None (the long way refuses it),
    and a wrong number of arguments is an error."""
    import torch

    import moe_grouped_matrix_amd as m
    from moe_grouped_matrix_amd import _moe, build
    if not os.path.exists(m.LIB_PATH) or not os.path.exists(_moe.EXT_PATH):
        build.build()
    ext = _moe._load_ext()
    ids, x = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 64, dtype=torch.bfloat16)
    slots = torch.zeros(4, 2, dtype=torch.int32)
    assert ext.sort_tokens(ids, 4, 0) is None and ext.sort_tokens(None, 4, 0) is None
    assert ext.dispatch(x, slots, 0) is None and ext.dispatch(x, "slots", 0) is None
    assert ext.combine(x, slots, None, -1, 0) is None
    assert ext.combine_grad(x, x, slots, None, 0) is None
    assert ext.quant_mxfp4(x, 2, 0) is None and ext.widen_mxfp4(x, x, 2, 1, 0) is None
    assert ext.sort_tokens(ids, "four", 0) is None and ext.sort_tokens(ids, 1 << 70, 0) is None
    for call_ in (lambda: ext.dispatch(x), lambda: ext.bind(1), lambda: ext.set_handle(0)):
        with pytest.raises(TypeError):
            call_()
    assert m.EXPORTED_MOE[0] == "gmm_sort_tokens_workspace" and len(m.EXPORTED_MOE) == 7


def test_binding_packs_the_c_struct():
    """The packed bytes are the ctypes structure's, field by field."""
    import torch

    from moe_grouped_matrix_amd import _binding, _moe
    s = _moe._TENSOR.pack(0x123450, 7, 3, 5, 6, 7, 0)
    t = _binding.GmmTensor.from_buffer_copy(s)
    assert (t.data, t.dtype, t.ndim, list(t.shape)) == (0x123450, 7, 3, [5, 6, 7, 0])
    with pytest.raises(_binding.GmmInvalid, match="device tensor"):
        _moe._pack(torch.zeros(2), "x", torch.device("cuda", 0))
    with pytest.raises(_binding.GmmInvalid, match="device tensor"):
        _moe._pack(None, "x", torch.device("cuda", 0))
