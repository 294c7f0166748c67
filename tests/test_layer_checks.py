"""Refusals of the entry points of include/gmm_layer.h on the CPU: the argument
checks are plain host C++, compiled here with the C++ compiler and called
through ctypes (no GPU, no library); the header against the library's exports;
and the step's factors, which the host and the device compute alike."""
import ctypes
import math
import os
import re
import subprocess

import pytest

from test_moe_checks import (A, B, BF16, C, CXX, D, E, E4M3, E8M0, F, F32, F4, I4, I8, I32, I64, INVALID, OK, ROOT, U4,
                             UNSUPPORTED, Tensor, call, good, refused, tensor)

SOURCE = r"""
#include "gmm_layer_checks.hpp"
using namespace gmmh;
typedef const gmm_tensor* T;
static thread_local std::string text;
static int say(const Check& c) { text = c.text; return c.status; }
extern "C" {
const char* why() { return text.c_str(); }
int route(T l, T b, T v, int s, T i, T w) { return say(check_route(l, b, v, s, i, w)); }
int balance(T l, T i, T v, int s, T o, T c, T n, const void* w, size_t b) { return say(check_balance_loss(l, i, v, s, o, c, n, w, b)); }
int grad(T l, T i, T v, int s, T dw, T c, T n, T dl, T o) { return say(check_router_grad(l, i, v, s, dw, c, n, dl, o)); }
int gmv(T x, T r, T s, T z, T i, T w, T o, const void* ws, size_t b) { return say(check_gmv(x, r, s, z, i, w, o, ws, b)); }
int adamw(const gmm_adamw_item* items, long long n, const gmm_adamw_args* a) { return say(check_adamw(items, n, a)); }
long long balance_bytes(long long t, long long e) { return (long long)balance_workspace_bytes(t, e); }
int item_size() { return (int)sizeof(gmm_adamw_item); }
int args_size() { return (int)sizeof(gmm_adamw_args); }
}
"""

H, I, J = ((i + 1) << 40 for i in range(6, 9))  # more addresses, far apart


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
    so.balance_bytes.restype = ctypes.c_longlong
    return so


P = ctypes.c_void_p


def swapped(args, **kw):
    """The arguments with those at the given places (a0, a1, ...) replaced."""
    args = list(args)
    for name, v in kw.items():
        args[int(name[1:])] = v
    return args


def test_route(lib):
    ok = [tensor(A, F32, 5, 16), None, None, 0, tensor(B, I32, 5, 4), tensor(C, F32, 5, 4)]
    good(lib, "route", *ok)
    good(lib, "route", *swapped(ok, a0=tensor(A, BF16, 5, 16), a1=tensor(D, F32, 16), a2=tensor(E, I8, 5), a3=1))
    good(lib, "route", tensor(None, F32, 0, 16), None, None, 0, tensor(None, I32, 0, 4), tensor(None, F32, 0, 4))
    good(lib, "route", tensor(A, F32, 5, 1024), None, None, 0, tensor(B, I32, 5, 64), tensor(C, F32, 5, 64))
    for status, word, kw in (
            (INVALID, "required", dict(a0=None)), (INVALID, "required", dict(a5=None)),
            (INVALID, "f32 or bf16", dict(a0=tensor(A, I32, 5, 16))), (INVALID, "(T, E)", dict(a0=tensor(A, F32, 80))),
            (INVALID, "(T, E)", dict(a0=tensor(A, F32, 5, 0))), (UNSUPPORTED, "1024 experts", dict(a0=tensor(A, F32, 5, 1025))),
            (UNSUPPORTED, "2^31", dict(a0=tensor(A, F32, 1 << 28, 16), a4=tensor(B, I32, 1 << 28, 4))),
            (UNSUPPORTED, "2^31", dict(a0=tensor(A, F32, 1 << 62, 16))),
            (INVALID, "int32", dict(a4=tensor(B, I64, 5, 4))), (INVALID, "k >= 1", dict(a4=tensor(B, I32, 5, 0))),
            (UNSUPPORTED, "64 choices", dict(a0=tensor(A, F32, 5, 128), a4=tensor(B, I32, 5, 65))),
            (INVALID, "more choices than experts", dict(a4=tensor(B, I32, 5, 17))), (INVALID, "differ", dict(a4=tensor(B, I32, 6, 4))),
            (INVALID, "valid", dict(a2=tensor(E, I8, 6))), (INVALID, "valid", dict(a2=tensor(E, F32, 5))),
            (INVALID, "scores", dict(a3=2)), (INVALID, "bias", dict(a1=tensor(D, BF16, 16))), (INVALID, "bias", dict(a1=tensor(D, F32, 15))),
            (INVALID, "weights", dict(a5=tensor(C, BF16, 5, 4))), (INVALID, "weights", dict(a5=tensor(C, F32, 4, 5))),
            (INVALID, "null", dict(a0=tensor(None, F32, 5, 16))), (INVALID, "16-byte", dict(a4=tensor(B + 4, I32, 5, 4))),
            (INVALID, "overlaps an input", dict(a4=tensor(A + 16, I32, 5, 4))), (INVALID, "two outputs", dict(a5=tensor(B, F32, 5, 4)))):
        refused(lib, status, word, "route", *swapped(ok, **kw))


def test_balance_loss(lib):
    need = lib.balance_bytes(ctypes.c_longlong(500), ctypes.c_longlong(16))
    ok = [tensor(A, F32, 500, 16), tensor(B, I64, 500, 4), None, 0, tensor(C, F32, 1), tensor(D, I32, 16), tensor(E, I32, 1),
          P(F), ctypes.c_size_t(need)]
    good(lib, "balance", *ok)
    good(lib, "balance", *swapped(ok, a1=tensor(B, I32, 500, 4), a2=tensor(H, I8, 500)))
    # one workgroup needs none
    assert lib.balance_bytes(ctypes.c_longlong(64), ctypes.c_longlong(16)) == 0 == lib.balance_bytes(ctypes.c_longlong(0), ctypes.c_longlong(1024))
    good(lib, "balance", *swapped(ok, a0=tensor(A, F32, 64, 16), a1=tensor(B, I64, 64, 4), a7=P(None), a8=ctypes.c_size_t(0)))
    for status, word, kw in (
            (INVALID, "required", dict(a6=None)), (INVALID, "int32 or int64", dict(a1=tensor(B, F32, 500, 4))),
            (INVALID, "loss", dict(a4=tensor(C, F32, 2))), (INVALID, "loss", dict(a4=tensor(C, BF16, 1))),
            (INVALID, "counts", dict(a5=tensor(D, I32, 15))), (INVALID, "tokens", dict(a6=tensor(E, I64, 1))),
            (INVALID, "overlaps an input", dict(a5=tensor(A, I32, 16))), (INVALID, "two outputs", dict(a6=tensor(D, I32, 1))),
            (INVALID, "workspace needs", dict(a7=P(None))), (INVALID, "workspace needs", dict(a8=ctypes.c_size_t(need - 1))),
            (INVALID, "16-byte", dict(a7=P(F + 4))), (INVALID, "workspace overlaps", dict(a7=P(D)))):
        refused(lib, status, word, "balance", *swapped(ok, **kw))


def test_router_grad(lib):
    ok = [tensor(A, BF16, 5, 16), tensor(B, I32, 5, 4), None, 1, tensor(C, F32, 5, 4), tensor(D, I32, 16), tensor(E, I32, 1),
          tensor(F, F32, 1), tensor(H, BF16, 5, 16)]
    good(lib, "grad", *ok)
    good(lib, "grad", *swapped(ok, a4=None, a7=None))
    good(lib, "grad", *swapped(ok, a4=tensor(C, BF16, 5, 4), a5=None, a6=None, a7=None))
    for status, word, kw in (
            (INVALID, "required", dict(a8=None)), (INVALID, "no gradient", dict(a4=None, a5=None, a6=None, a7=None)),
            (INVALID, "come together", dict(a6=None)), (INVALID, "come together", dict(a5=None)),
            (INVALID, "dloss without", dict(a5=None, a6=None)), (INVALID, "dweights", dict(a4=tensor(C, F32, 4, 5))),
            (INVALID, "dweights", dict(a4=tensor(C, I32, 5, 4))), (INVALID, "counts", dict(a5=tensor(D, I32, 17))),
            (INVALID, "tokens", dict(a6=tensor(E, F32, 1))), (INVALID, "dloss", dict(a7=tensor(F, F32, 2))),
            (INVALID, "dlogits", dict(a8=tensor(H, F32, 5, 16))), (INVALID, "dlogits", dict(a8=tensor(H, BF16, 16, 5))),
            (INVALID, "overlaps an input", dict(a8=tensor(A, BF16, 5, 16)))):
        refused(lib, status, word, "grad", *swapped(ok, **kw))


def gmv_args(T=3, k=2, G=5, N=24, K=64, nb=2):
    return [tensor(A, BF16, T, K), tensor(B, I4, G, N, K), tensor(C, F32, G, nb, 1, N), tensor(D, F32, G, nb, 1, N),
            tensor(E, I32, T, k), None, tensor(F, F32, T, k, N), P(None), ctypes.c_size_t(0)]


def test_gmv(lib):
    ok = gmv_args()
    good(lib, "gmv", *ok)
    good(lib, "gmv", *swapped(ok, a0=tensor(A, BF16, 3, 2, 64), a1=tensor(B, U4, 5, 24, 64), a4=tensor(E, I64, 3, 2)))
    good(lib, "gmv", *swapped(ok, a2=tensor(C, BF16, 5, 1, 1, 24), a3=tensor(D, BF16, 5, 1, 1, 24)))
    good(lib, "gmv", *swapped(ok, a1=tensor(B, F4, 5, 24, 64), a2=tensor(C, E8M0, 5, 2, 1, 24), a3=None))
    few = swapped(ok, a5=tensor(H, F32, 3, 2), a6=tensor(F, BF16, 3, 24))  # (no workspace)
    good(lib, "gmv", *few)
    weighted = swapped(gmv_args(T=9), a5=tensor(H, F32, 9, 2), a6=tensor(F, BF16, 9, 24), a7=P(I), a8=ctypes.c_size_t(9 * 2 * 24 * 4))
    good(lib, "gmv", *weighted)
    dense = swapped(gmv_args(T=7, k=1, G=1), a4=None)
    good(lib, "gmv", *dense)
    good(lib, "gmv", *swapped(dense, a0=tensor(None, BF16, 0, 64), a6=tensor(None, F32, 0, 1, 24)))
    good(lib, "gmv", *gmv_args(T=4096, k=1))
    for status, word, kw in (
            (INVALID, "required", dict(a2=None)), (INVALID, "x must be bf16", dict(a0=tensor(A, F32, 3, 64))),
            (INVALID, "int4, uint4", dict(a1=tensor(B, I8, 5, 24, 64))), (INVALID, "(G, N, K)", dict(a1=tensor(B, I4, 24, 64))),
            (INVALID, "(G, N, K)", dict(a1=tensor(B, I4, 5, 0, 64))), (UNSUPPORTED, "1024 groups", dict(a1=tensor(B, I4, 1025, 24, 64))),
            (INVALID, "multiple of 32", dict(a1=tensor(B, I4, 5, 24, 48))), (UNSUPPORTED, "2^20", dict(a1=tensor(B, I4, 5, 24, 1 << 20))),
            (UNSUPPORTED, "2^24", dict(a1=tensor(B, I4, 5, 1 << 24, 64))), (INVALID, "int32 or int64", dict(a4=tensor(E, F32, 3, 2))),
            (INVALID, "expert_ids are required", dict(a4=None)), (UNSUPPORTED, "64 choices", dict(a4=tensor(E, I32, 3, 65))),
            (UNSUPPORTED, "4096 slots", dict(a4=tensor(E, I32, 2049, 2))), (INVALID, "x of shape", dict(a0=tensor(A, BF16, 4, 64))),
            (INVALID, "x of shape", dict(a0=tensor(A, BF16, 3, 3, 64))), (INVALID, "x of shape", dict(a0=tensor(A, BF16, 3, 32))),
            (INVALID, "rhs_scale", dict(a2=tensor(C, F32, 5, 2, 24))), (INVALID, "rhs_scale", dict(a2=tensor(C, F32, 5, 2, 1, 25))),
            (INVALID, "K/nb", dict(a2=tensor(C, F32, 5, 4, 1, 24))), (INVALID, "K/nb", dict(a2=tensor(C, F32, 5, 3, 1, 24))),
            (INVALID, "K/nb", dict(a2=tensor(C, F32, 5, 1 << 40, 1, 24))), (INVALID, "rhs_scale", dict(a2=tensor(C, F32, 5, 0, 1, 24))),
            (INVALID, "E8M0", dict(a2=tensor(C, E8M0, 5, 2, 1, 24), a3=None)), (INVALID, "f32, bf16 or E8M0", dict(a2=tensor(C, I8, 5, 2, 1, 24))),
            (INVALID, "E8M0", dict(a1=tensor(B, F4, 5, 24, 64), a2=tensor(C, E8M0, 5, 1, 1, 24), a3=None)),
            (INVALID, "no zero points", dict(a1=tensor(B, F4, 5, 24, 64))), (INVALID, "rhs_zero", dict(a3=tensor(D, BF16, 5, 2, 1, 24))),
            (INVALID, "rhs_zero", dict(a3=tensor(D, F32, 5, 1, 1, 24))), (INVALID, "out", dict(a6=tensor(F, I32, 3, 2, 24))),
            (INVALID, "(T, k, N)", dict(a6=tensor(F, F32, 3, 24))), (INVALID, "overlaps an input", dict(a6=tensor(A, F32, 3, 2, 24))),
            (INVALID, "null", dict(a0=tensor(None, BF16, 3, 64))), (INVALID, "16-byte", dict(a1=tensor(B + 8, I4, 5, 24, 64)))):
        refused(lib, status, word, "gmv", *swapped(ok, **kw))
    for status, word, kw in ((INVALID, "(T, N)", dict(a6=tensor(F, BF16, 9, 2, 24))), (INVALID, "weights", dict(a5=tensor(H, F32, 2, 9))),
                             (INVALID, "weights", dict(a5=tensor(H, I32, 9, 2))), (INVALID, "workspace needs", dict(a7=P(None))),
                             (INVALID, "workspace overlaps", dict(a7=P(F))), (INVALID, "16-byte", dict(a7=P(I + 4)))):
        refused(lib, status, word, "gmv", *swapped(weighted, **kw))


class Item(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64)] + [(n, P) for n in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                                             "exp_avg_sq_scale", "copy")]


class Args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("param_dtype", "grad_dtype", "state_dtype")] +
                [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] +
                [("step", ctypes.c_int64)] + [(n, P) for n in ("step_at", "lr_at", "grad_scale")])


def adam(lib, status, word, items, **kw):
    fields = dict(param_dtype=F32, grad_dtype=BF16, state_dtype=F32, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1)
    args = Args(**dict(fields, **kw))
    array = (Item * max(1, len(items)))(*items)
    got = lib.adamw(array, ctypes.c_longlong(len(items)), ctypes.byref(args))
    text = lib.why().decode()
    assert got == status and word in text, (got, text)


def test_adamw(lib):
    from moe_grouped_matrix_amd import _layer
    assert lib.item_size() == ctypes.sizeof(Item) == _layer._ITEM.size
    assert lib.args_size() == ctypes.sizeof(Args) == _layer._ARGS.size
    item = lambda n=1000, at=0, **kw: Item(**dict(dict(n=n, param=A + at, grad=B + at, exp_avg=C + at, exp_avg_sq=D + at), **kw))  # noqa: E731
    eight = lambda n=1000, at=0, **kw: item(n, at, **dict(dict(exp_avg_scale=E + at, exp_avg_sq_scale=F + at), **kw))  # noqa: E731
    adam(lib, OK, "", [])
    adam(lib, OK, "", [item()])
    adam(lib, OK, "", [item(at=1 << 20), item(copy=H), item(0, param=None)])  # (in any order)
    adam(lib, OK, "", [eight(at=4096 * i) for i in range(100)], state_dtype=E4M3)
    adam(lib, OK, "", [item(), item(at=1 << 20, grad=B)])  # gradients may be one
    adam(lib, OK, "", [item()], step=0, step_at=H, lr_at=I, grad_scale=J)
    args = Args(param_dtype=F32, grad_dtype=F32, state_dtype=F32, step=1)
    for got in (lib.adamw(None, ctypes.c_longlong(1), ctypes.byref(args)), lib.adamw(None, ctypes.c_longlong(-1), ctypes.byref(args)),
                lib.adamw(None, ctypes.c_longlong(0), None)):
        assert got == INVALID and "required" in lib.why().decode()
    for word, kw in (("parameters and gradients", dict(param_dtype=I32)), ("parameters and gradients", dict(grad_dtype=E4M3)),
                     ("states must be", dict(state_dtype=BF16)), ("lr must", dict(lr=-1.0)), ("lr must", dict(lr=math.nan)),
                     ("lr must", dict(lr=math.inf)), ("betas", dict(beta1=1.0)), ("betas", dict(beta2=-0.1)), ("betas", dict(beta2=math.nan)),
                     ("eps must", dict(eps=-1e-8)), ("eps must", dict(eps=math.nan)), ("weight_decay", dict(weight_decay=-0.1)),
                     ("counted from 1", dict(step=0)), ("4-byte", dict(lr_at=H + 2)), ("overlaps a tensor", dict(step_at=A + 16))):
        adam(lib, INVALID, word, [item()], **kw)
    for word, items in (("tensor 1: negative", [item(), item(-1)]), ("null", [item(param=None)]), ("null", [item(grad=None)]),
                        ("f32 states have no scales", [eight()]), ("16-byte", [item(exp_avg=C + 4)]), ("16-byte", [item(copy=H + 8)]),
                        ("overlap", [item(), item()]), ("overlap", [item(), item(at=3984)]), ("overlap", [item(exp_avg=A + 3984)]),
                        ("overlap", [item(copy=D)]), ("gradient overlaps", [item(grad=C + 3984)]), ("gradient overlaps", [item(grad=C - 1984)])):
        adam(lib, INVALID, word, items)
    adam(lib, OK, "", [item(), item(at=4000, grad=B + 4000)])
    adam(lib, OK, "", [item(grad=C + 4000)])
    adam(lib, UNSUPPORTED, "2^34", [item(1 << 34)])
    adam(lib, INVALID, "need scales", [item()], state_dtype=E4M3)
    adam(lib, INVALID, "need scales", [eight(exp_avg_sq_scale=None)], state_dtype=E4M3)
    adam(lib, INVALID, "overlap", [eight(), eight(at=1 << 20, exp_avg_scale=E)], state_dtype=E4M3)


def declared():
    text = open(os.path.join(ROOT, "include", "gmm_layer.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*gmm_status\s+(gmm_\w+)\s*\(", text, flags=re.M)


def test_library_exports_the_header():
    import moe_grouped_matrix_amd as m
    from moe_grouped_matrix_amd import _binding, build
    if not os.path.exists(_binding.LIB_PATH):
        build.build()
    lib = m.load()
    assert sorted(declared()) == sorted(m.EXPORTED_LAYER)
    for name in m.EXPORTED_LAYER:
        assert hasattr(lib, name), name
    text = open(os.path.join(ROOT, "include", "gmm_layer.h")).read()
    assert "#define GMM_ADAMW_BLOCK %d\n" % m.ADAMW_BLOCK in text
    assert "#define GMM_SCORES_SOFTMAX 0\n" in text and "#define GMM_SCORES_SIGMOID 1\n" in text
    need = ctypes.c_size_t(7)
    assert lib.gmm_gmv_workspace(8, 1408, 0, ctypes.byref(need)) == OK and need.value == 0
    assert lib.gmm_gmv_workspace(8, 1408, 1, ctypes.byref(need)) == OK and need.value == 0
    assert lib.gmm_gmv_workspace(80, 1408, 1, ctypes.byref(need)) == OK and need.value == 80 * 1408 * 4
    assert lib.gmm_gmv_workspace(4097, 1408, 1, ctypes.byref(need)) == UNSUPPORTED
    assert lib.gmm_gmv_workspace(-1, 1408, 1, ctypes.byref(need)) == INVALID
    assert lib.gmm_balance_loss_workspace(32768, 128, ctypes.byref(need)) == OK and need.value < 1 << 20
    assert lib.gmm_balance_loss_workspace(1 << 31, 1, ctypes.byref(need)) == UNSUPPORTED
    assert lib.gmm_balance_loss_workspace(5, 0, ctypes.byref(need)) == INVALID
