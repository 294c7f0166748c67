"""The compiled binding of the operators of gmm_layer.h (csrc/moe_ext.cpp) on
the CPU: the file is compiled so that host tensors pass for tensors of device
0, and bound to entry points that take down their arguments.  What it hands to
the library has to be what the Python marshalling (_layer.py) hands over for
the same call; everything that it does not take comes back as None."""
import ctypes
import importlib.util
import os
import subprocess

import pytest
import torch

from moe_grouped_matrix_amd import _binding, _layer, _moe, build
from test_moe_ext_host import dev, fields
from test_stream_argument import Device

SOURCE = r"""
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>
#include <cstring>
#include "gmm_layer.h"
#include "gmm_moe.h"
// a host tensor is one of device 0
#define is_cuda is_cpu
#define get_device() dim() * 0
#include "moe_ext.cpp"
#undef is_cuda
#undef get_device

static gmm_tensor g_taken[8];
static double g_numbers[8];
static int g_count, g_nums;
static std::vector<gmm_adamw_item> g_items;
static gmm_adamw_args g_args;
static gmm_status take(std::initializer_list<const gmm_tensor*> ts, std::initializer_list<double> ns) {
  g_count = g_nums = 0;
  for (const gmm_tensor* t : ts) {
    if (t) g_taken[g_count] = *t;
    else std::memset(&g_taken[g_count], 0, sizeof(gmm_tensor));
    ++g_count;
  }
  for (double v : ns) g_numbers[g_nums++] = v;
  return GMM_OK;
}
extern "C" {
typedef const gmm_tensor* T;
gmm_status rec_route(gmm_handle*, T a, T b, T c, int s, int r, float f, T d, T e, void* st) {
  return take({a, b, c, d, e}, {(double)s, (double)r, f, (double)(uintptr_t)st});
}
gmm_status rec_space(int64_t, int64_t, size_t* n) { *n = 64; return GMM_OK; }
gmm_status rec_balance(gmm_handle*, T a, T b, T c, int s, float f, float z, T d, T e, T g, void* w, size_t n, void* st) {
  return take({a, b, c, d, e, g}, {(double)s, f, z, w ? 1. : 0., (double)n, (double)(uintptr_t)st});
}
gmm_status rec_grad(gmm_handle*, T a, T b, T c, int s, T d, int r, float f, T e, T g, T h, float x, float z, T o, void* st) {
  return take({a, b, c, d, e, g, h, o}, {(double)s, (double)r, f, x, z, (double)(uintptr_t)st});
}
gmm_status rec_gmv_space(int64_t, int64_t, int w, size_t* n) { *n = w ? 64 : 0; return GMM_OK; }
gmm_status rec_gmv(gmm_handle*, T a, T b, T c, T d, T e, T f, T o, void* w, size_t n, void* st) {
  return take({a, b, c, d, e, f, o}, {w ? 1. : 0., (double)n, (double)(uintptr_t)st});
}
gmm_status rec_adamw(gmm_handle*, const gmm_adamw_item* items, int64_t n, const gmm_adamw_args* a, void* st) {
  g_items.assign(items, items + n);
  g_args = *a;
  return take({}, {(double)(uintptr_t)st});
}
int rec_get(gmm_tensor* out, double* numbers, int* nums) {
  std::memcpy(out, g_taken, sizeof g_taken);
  std::memcpy(numbers, g_numbers, sizeof g_numbers);
  *nums = g_nums;
  return g_count;
}
int rec_step(void* items, void* args) {
  std::memcpy(items, g_items.data(), g_items.size() * sizeof(gmm_adamw_item));
  std::memcpy(args, &g_args, sizeof g_args);
  return (int)g_items.size();
}
}
"""
ENTRIES = ("rec_route", "rec_space", "rec_balance", "rec_grad", "rec_gmv_space", "rec_gmv", "rec_adamw")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("ext")
    (d / "t.cpp").write_text(SOURCE)
    so = str(d / "_moe_ext.so")
    cmd = build._ext_command(so)
    cmd[cmd.index(os.path.join(build.CSRC, "moe_ext.cpp"))] = str(d / "t.cpp")
    cmd[cmd.index("-O2")] = "-O0"
    subprocess.run(cmd + ["-I" + build.CSRC], check=True)
    spec = importlib.util.spec_from_file_location("_moe_ext", so)
    ext = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ext)
    c = ctypes.CDLL(so)
    ext.bind_layer(*[ctypes.cast(getattr(c, name), ctypes.c_void_p).value for name in ENTRIES])
    ext.set_handle(0, 0x1000)
    return ext, c


def taken(c):
    buf, numbers, nums = (_binding.GmmTensor * 8)(), (ctypes.c_double * 8)(), ctypes.c_int()
    n = c.rec_get(buf, numbers, ctypes.byref(nums))
    return [fields(buf[i]) for i in range(n)], list(numbers)[:nums.value]


class Asked:
    """Stands in for the extension in the binding: takes down what it is asked
    and leaves the call to Python."""

    def __init__(self):
        self.asked = None

    def set_handle(self, *_):
        pass

    def __getattr__(self, name):
        def ask(*args):
            self.asked = name, args
        return ask


@pytest.fixture
def python_way(monkeypatch):
    """calls(fn) -> (what the extension was asked, what Python handed to the library, its outputs)"""
    seen, asked = [], Asked()

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name == "gmm_balance_loss_workspace" or name == "gmm_gmv_workspace" and args[2]:
                    args[-1]._obj.value = 64
                elif not name.endswith("workspace"):
                    seen[:] = args[1:]
                return 0
            return call

    empty, strided = torch.empty, torch.empty_strided
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw).as_subclass(Device))
    monkeypatch.setattr(torch, "empty_strided", lambda *a, device=None, **kw: strided(*a, **kw).as_subclass(Device))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x77, raising=False)
    monkeypatch.setattr(_layer, "_current", lambda t: 0x77)
    monkeypatch.setattr(_binding, "_lib", Library())
    monkeypatch.setattr(_binding, "_handles", {0: 1})
    monkeypatch.setattr(_moe, "_ext", asked)
    for cached in (_layer._balance_workspace, _layer._gmv_workspace):
        cached.cache_clear()

    def calls(fn):
        outs = fn()
        return asked.asked, list(seen), outs if isinstance(outs, tuple) else (outs,)
    yield calls
    for cached in (_layer._balance_workspace, _layer._gmv_workspace):
        cached.cache_clear()


F32, BF16, I32, I64, U8, I8, E8, E4 = (torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8, torch.int8,
                                       torch.float8_e8m0fnu, torch.float8_e4m3fn)


def cases():
    for T in (0, 5):
        ids, valid = {d: dev(T, 3, dtype=d) for d in (I32, I64)}, [None] + [dev(T, dtype=d) for d in (torch.bool, U8, I8)]
        dw, counts, one = dev(T, 3, dtype=BF16), dev(16, dtype=I32), dev(1, dtype=I32)
        for z in (dev(T, 16, dtype=F32), dev(T, 16, dtype=BF16)):
            for v in valid:
                yield lambda z=z, v=v: _layer.route(z, 3, valid=v)
                yield lambda z=z, v=v: _layer.route(z, 3, scores="sigmoid", bias=dev(16, dtype=F32), renormalize=False, scale=2.5, valid=v)
                for d in ids:
                    yield lambda z=z, v=v, d=d: _layer.balance_loss(z, ids[d], scores="sigmoid", coef=0.5, z_coef=0.25, valid=v)
                    yield lambda z=z, v=v, d=d: _layer.router_grad(z, ids[d], dweights=dw, valid=v, renormalize=False, scale=4)
                    yield lambda z=z, v=v, d=d: _layer.router_grad(z, ids[d], dweights=dev(T, 3, dtype=F32), scores="sigmoid", counts=counts,
                                                                   tokens=one, dloss=dev(1, dtype=F32), coef=0.5, z_coef=0.125, valid=v)
        q, s, z = dev(4, 24, 32, dtype=U8), dev(4, 2, 1, 24, dtype=F32), dev(4, 2, 1, 24, dtype=F32)
        for x in (dev(T, 64, dtype=BF16), dev(T, 3, 64, dtype=BF16)):
            for i in (ids[I32], ids[I64], None):
                for w in (None, dev(T, 3, dtype=F32), dev(T, 3, dtype=BF16)):
                    for out in (F32, BF16):
                        yield lambda x=x, i=i, w=w, out=out: _layer.gmv(x, q, i, rhs_format="int4", rhs_scale=s, rhs_zero=z, weights=w, out_dtype=out)
        yield lambda: _layer.gmv(dev(T, 64, dtype=BF16), q, ids[I32], rhs_format="fp4_e2m1", rhs_scale=dev(4, 2, 1, 24, dtype=E8))
        yield lambda: _layer.gmv(dev(T, 64, dtype=BF16), q, ids[I32], rhs_format="uint4", rhs_scale=dev(4, 2, 1, 24, dtype=BF16))


def test_both_ways_hand_over_the_same(host, python_way):
    ext, c = host
    count = 0
    for call in cases():
        (name, args), seen, outs = python_way(call)
        made = getattr(ext, name)(*args)
        assert made is not None, (name, args)
        made = made if isinstance(made, tuple) else (made,)
        views, numbers = taken(c)
        want, wnum = [], []
        for a in seen:
            if isinstance(a, bytes):
                want.append(fields(_binding.GmmTensor.from_buffer_copy(a)))
            elif a is None and len(want) < len(views):
                want.append((False, 0, 0, ()))
            elif a is not None:
                wnum.append(a)
        strip = lambda vs: [(d and 0 not in s, *r, s) for d, *r, s in vs]  # noqa: E731
        assert strip(views) == strip(want), name
        if name in ("balance_loss", "gmv"):  # (an address of the workspace, or none)
            at = -3
            assert bool(numbers[at]) == bool(numbers[at + 1])
            numbers.pop(at)
            if len(wnum) > len(numbers):
                wnum.pop(at)
        assert numbers == [float(torch.tensor(float(v), dtype=F32)) if isinstance(v, float) else v for v in wnum], name
        assert [(tuple(a.shape), a.dtype) for a in made] == [(tuple(b.shape), b.dtype) for b in outs], name
        count += 1
    assert count == 2 * (2 * 4 * (2 + 2 * 3) + 2 * 3 * 3 * 2 + 2)


def test_both_ways_hand_over_the_same_step(host, python_way):
    ext, c = host
    for eight in (False, True):
        for many in (1, 70):
            st = E4 if eight else F32
            col = lambda d, n=600: [dev(n, dtype=d) for _ in range(many)]  # noqa: E731
            for copies, lists in ((None, list), (col(BF16), tuple)):
                kw = dict(exp_avg_scale=lists(col(F32, 3)), exp_avg_sq_scale=lists(col(F32, 3))) if eight else {}
                for step, lr, gs in ((7, 0.5, None), (dev(1, dtype=I32), dev(1, dtype=F32), dev(1, dtype=F32))):
                    (name, args), seen, _ = python_way(lambda: _layer.adamw(
                        lists(col(F32)), lists(col(BF16)), lists(col(st)), lists(col(st)), step, lr=lr, betas=(0.25, 0.125), eps=2.0,
                        weight_decay=4.0, copies=copies, grad_scale=gs, **kw))
                    items, n, want, stream = seen
                    assert getattr(ext, name)(*args) is True
                    got, gargs = ctypes.create_string_buffer(many * _layer._ITEM.size), ctypes.create_string_buffer(_layer._ARGS.size)
                    assert c.rec_step(got, gargs) == n == many and taken(c)[1] == [0x77] == [stream]
                    assert got.raw == items
                    assert _layer._ARGS.unpack(gargs.raw) == _layer._ARGS.unpack(want)


def test_other_forms_go_the_long_way(host):
    ext, c = host
    z, ids, w = dev(4, 16, dtype=F32), dev(4, 3, dtype=I32), dev(4, 3, dtype=F32)
    x, q, s = dev(4, 64, dtype=BF16), dev(4, 24, 32, dtype=U8), dev(4, 2, 1, 24, dtype=F32)
    good = [("route", (z, 3, None, None, 0, True, 1.0, 0x77)), ("balance_loss", (z, ids, None, 0, 1.0, 0.0, 0x77)),
            ("router_grad", (z, ids, None, 0, w, True, 1.0, None, None, None, 1.0, 0.0, 0x77)),
            ("gmv", (x, q, 7, s, None, ids, None, 0, 0x77)),
            ("adamw", ([z], [z], [z], [z], None, None, None, 1, 0.1, 0.9, 0.99, 1e-8, 0.0, None, 0x77))]
    bad = [("route", {0: z[0]}), ("route", {0: z.t()}), ("route", {1: 17}), ("route", {1: 0}), ("route", {3: dev(4, dtype=F32)}),
           ("route", {6: "x"}), ("route", {7: "s"}), ("balance_loss", {1: w}), ("balance_loss", {2: 3}), ("balance_loss", {4: None}),
           ("router_grad", {1: ids[0]}), ("router_grad", {4: "w"}), ("gmv", {0: x[0]}), ("gmv", {1: dev(4, 24, 32, dtype=I8)}),
           ("gmv", {5: w}), ("gmv", {7: 3}), ("gmv", {3: None}), ("adamw", {0: []}), ("adamw", {0: z}), ("adamw", {1: [z, z]}),
           ("adamw", {1: [dev(3, dtype=F32)]}), ("adamw", {1: [None]}), ("adamw", {3: [dev(4, 16, dtype=E4)]}), ("adamw", {4: [z]}),
           ("adamw", {6: [z]}), ("adamw", {7: dev(1, dtype=I64)}), ("adamw", {8: dev(2, dtype=F32)}), ("adamw", {8: "x"}),
           ("adamw", {13: 0.5}), ("adamw", {0: [z.t()]})]
    for name, args in good:
        assert getattr(ext, name)(*args) is not None, name
    for name, change in bad:
        args = list(dict(good)[name])
        for i, v in change.items():
            args[i] = v
        assert getattr(ext, name)(*args) is None, (name, change)
