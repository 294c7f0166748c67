"""The compiled binding (csrc/moe_ext.cpp) on the CPU: the file is compiled so
that host tensors pass for tensors of device 0, and bound to entry points that
take down their arguments instead of queueing work.

What it hands to the library has to be what the Python marshalling (_moe.py)
hands over for the same call, over every type and form that either takes; and
other Python threads have to run while a call is queued."""
import ctypes
import importlib.util
import itertools
import os
import subprocess
import threading

import pytest
import torch

from moe_grouped_matrix_amd import _binding, _moe, build
from test_stream_argument import DEV, Device

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>
#include <atomic>
#include <chrono>
#include <cstring>
#include <thread>
#include "gmm_moe.h"
// a host tensor is one of device 0
#define is_cuda is_cpu
#define get_device() dim() * 0
#include "moe_ext.cpp"
#undef is_cuda
#undef get_device

static gmm_tensor g_taken[6];
static int g_count;
static void* g_stream;
static std::atomic<int> g_wait{0}, g_open{0};

// Takes the arguments down; with g_wait set, waits up to 5 s for g_open.
static gmm_status take(std::initializer_list<const gmm_tensor*> ts, void* stream) {
  g_count = 0;
  for (const gmm_tensor* t : ts) {
    if (t) g_taken[g_count] = *t;
    else std::memset(&g_taken[g_count], 0, sizeof(gmm_tensor));
    ++g_count;
  }
  g_stream = stream;
  for (int i = 0; g_wait && i < 5000; ++i) {
    if (g_open) return GMM_OK;
    std::this_thread::sleep_for(std::chrono::milliseconds(1));
  }
  return g_wait ? GMM_E_INVALID : GMM_OK;
}

extern "C" {
typedef const gmm_tensor* T;
gmm_status rec_workspace(int64_t slots, int64_t groups, size_t* bytes) {
  *bytes = slots > 4096 ? 4096 : 0;
  return groups > 1024 ? GMM_E_UNSUPPORTED : GMM_OK;
}
gmm_status rec_sort(gmm_handle*, T a, T b, T c, void*, size_t, void* s) { return take({a, b, c}, s); }
gmm_status rec_dispatch(gmm_handle*, T a, T b, T c, void* s) { return take({a, b, c}, s); }
gmm_status rec_combine(gmm_handle*, T a, T b, T c, T d, void* s) { return take({a, b, c, d}, s); }
gmm_status rec_combine_grad(gmm_handle*, T a, T b, T c, T d, T e, T f, void* s) { return take({a, b, c, d, e, f}, s); }
gmm_status rec_three(gmm_handle*, T a, T b, T c, void* s) { return take({a, b, c}, s); }
void rec_gate(int wait, int open) { g_wait = wait; g_open = open; }
int rec_get(gmm_tensor* out, void** stream) {
  std::memcpy(out, g_taken, sizeof g_taken);
  *stream = g_stream;
  return g_count;
}
}
"""

ENTRIES = ("rec_workspace", "rec_sort", "rec_dispatch", "rec_combine", "rec_combine_grad", "rec_three", "rec_three")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """(the extension bound to the recording entry points, its C side)"""
    d = tmp_path_factory.mktemp("ext")
    (d / "t.cpp").write_text(SOURCE)
    so = str(d / "_moe_ext.so")
    cmd = build._ext_command(so)
    cmd[cmd.index(os.path.join(build.CSRC, "moe_ext.cpp"))] = str(d / "t.cpp")
    cmd[cmd.index("-O2")] = "-O0"
    subprocess.run(cmd + ["-I" + build.CSRC, "-pthread"], check=True)
    spec = importlib.util.spec_from_file_location("_moe_ext", so)
    ext = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ext)
    c = ctypes.CDLL(so)
    ext.bind(*[ctypes.cast(getattr(c, name), ctypes.c_void_p).value for name in ENTRIES])
    ext.set_handle(0, 0x1000)
    return ext, c


def fields(t):
    """A gmm_tensor without its address (kept as null or not)."""
    return bool(t.data), t.dtype, t.ndim, tuple(t.shape)[:t.ndim]


def taken(c):
    buf, stream = (_binding.GmmTensor * 6)(), ctypes.c_void_p()
    n = c.rec_get(buf, ctypes.byref(stream))
    return [fields(buf[i]) for i in range(n)], stream.value or 0


@pytest.fixture
def python_way(monkeypatch):
    """calls(fn) -> what the Python marshalling hands over, and its outputs."""
    seen = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name == "gmm_sort_tokens_workspace":
                    return 0
                seen[:] = [args[1:-1], args[-1]]
                return 0
            return call

    class Ext:
        def set_handle(self, *_):
            pass

        def __getattr__(self, name):
            return lambda *_: None

    empty, strided = torch.empty, torch.empty_strided
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw).as_subclass(Device))
    monkeypatch.setattr(torch, "empty_strided", lambda *a, device=None, **kw: strided(*a, **kw).as_subclass(Device))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x77, raising=False)
    # (a host tensor says device 0 of itself, but counts as none in C++)
    monkeypatch.setattr(_moe, "_current", lambda t: 0x77)
    monkeypatch.setattr(_binding, "_lib", Library())
    monkeypatch.setattr(_binding, "_handles", {0: 1})
    monkeypatch.setattr(_moe, "_ext", Ext())
    _moe._sort_workspace.cache_clear()

    def calls(fn):
        outs = fn()
        views = []
        for a in seen[0]:
            if isinstance(a, bytes):
                views.append(fields(_binding.GmmTensor.from_buffer_copy(a)))
            elif a is None:
                views.append((False, 0, 0, ()))
        return views, seen[1], outs if isinstance(outs, tuple) else (outs,)
    yield calls
    _moe._sort_workspace.cache_clear()


def dev(*shape, dtype):
    return torch.zeros(shape, dtype=torch.uint8).to(dtype).as_subclass(Device) if dtype not in (
        torch.float8_e8m0fnu,) else torch.zeros(shape, dtype=torch.uint8).view(dtype).as_subclass(Device)


F32, BF16, I32, I64, U8, E8 = (torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8,
                               torch.float8_e8m0fnu)


def cases():
    """(name, arguments of the extension, call of the Python binding)"""
    for T, dt in itertools.product((0, 1, 37), (I32, I64)):
        ids = dev(T, 3, dtype=dt)
        yield f"sort {T} {dt}", "sort_tokens", (ids, 9), lambda ids=ids: _moe.sort_tokens(ids, 9)
    for T in (0, 5):
        slots = dev(T, 3, dtype=I32)
        for dt in (F32, BF16, torch.float8_e4m3fn, torch.float8_e5m2, E8, torch.int8, U8, I32):
            x = dev(T, 64, dtype=dt)
            yield f"dispatch {T} {dt}", "dispatch", (x, slots), lambda x=x, s=slots: _moe.dispatch(x, s)
        for rd, wd, od in itertools.product((F32, BF16), (None, F32, BF16), (None, F32, BF16)):
            rows, w = dev(3 * T, 64, dtype=rd), None if wd is None else dev(T, 3, dtype=wd)
            code = -1 if od is None else _binding._DTYPE[od]
            yield (f"combine {T} {rd} {wd} {od}", "combine", (rows, slots, w, code),
                   lambda r=rows, s=slots, w=w, od=od: _moe.combine(r, s, w, out_dtype=od))
        for gd, rd, wd in itertools.product((F32, BF16), repeat=3):
            g, rows, w = dev(T, 64, dtype=gd), dev(3 * T, 64, dtype=rd), dev(T, 3, dtype=wd)
            yield (f"combine_grad {T} {gd} {rd} {wd}", "combine_grad", (g, rows, slots, w),
                   lambda g=g, r=rows, s=slots, w=w: _moe.combine_grad(g, r, s, w))
        for dt in (F32, BF16):
            x = dev(T, 96, dtype=dt)
            yield f"quant lhs {T} {dt}", "quant_mxfp4", (x, 2), lambda x=x: _moe.quant_mxfp4(x)
            x = dev(T, 7, 96, dtype=dt)
            yield f"quant rhs {T} {dt}", "quant_mxfp4", (x, 3), lambda x=x: _moe.quant_mxfp4(x, operand="rhs")
            q, e = dev(T, 48, dtype=U8), dev(T, 3, dtype=E8)
            yield (f"widen lhs {T} {dt}", "widen_mxfp4", (q, e, 2, _binding._DTYPE[dt]),
                   lambda q=q, e=e, dt=dt: _moe.widen_mxfp4(q, e, out_dtype=dt))
            q, e = dev(T, 7, 48, dtype=U8), dev(T, 3, 1, 7, dtype=E8)
            yield (f"widen rhs {T} {dt}", "widen_mxfp4", (q, e, 3, _binding._DTYPE[dt]),
                   lambda q=q, e=e, dt=dt: _moe.widen_mxfp4(q, e, operand="rhs", out_dtype=dt))


def test_both_ways_hand_over_the_same(host, python_way):
    ext, c = host
    count = 0
    for name, fn, args, call in cases():
        made = getattr(ext, fn)(*args, 0x77)
        assert made is not None, name
        made = made if isinstance(made, tuple) else (made,)
        views, stream = taken(c)
        want, wstream, outs = python_way(call)
        if fn == "sort_tokens":
            want = want[:3]  # (behind them comes the workspace)
        # (an address of an empty tensor is nobody's business)
        strip = [(d and 0 not in s, *r, s) for d, *r, s in views]
        assert strip == [(d and 0 not in s, *r, s) for d, *r, s in want], name
        assert stream == wstream == 0x77, name
        assert [(tuple(a.shape), a.dtype) for a in made] == [(tuple(b.shape), b.dtype) for b in outs], name
        count += 1
    assert count == 6 + 2 * (8 + 18 + 8 + 8)


def test_other_forms_go_the_long_way(host):
    """What the extension does not take comes back as None: other ranks, types,
    strides, numbers, and a refused call."""
    ext, c = host
    x, slots, ids = dev(4, 64, dtype=BF16), dev(4, 3, dtype=I32), dev(4, 3, dtype=I64)
    rows, w, q, e = dev(12, 64, dtype=BF16), dev(4, 3, dtype=F32), dev(4, 32, dtype=U8), dev(4, 2, dtype=E8)
    for fn, args in (("sort_tokens", (ids.t(), 9)), ("sort_tokens", (ids, 1025)), ("sort_tokens", (w, 9)),
                     ("sort_tokens", (ids, "9")), ("sort_tokens", (ids[0], 9)), ("dispatch", (x[:, ::2], slots)),
                     ("dispatch", (dev(4, 64, dtype=torch.float16), slots)), ("dispatch", (x, slots[0])),
                     ("combine", (rows, slots, w, -2)), ("combine", (rows, slots, "w", -1)),
                     ("combine", (rows, slots, w[0], -1)), ("combine_grad", (x, rows, slots, None)),
                     ("quant_mxfp4", (x, 3)), ("quant_mxfp4", (dev(4, 64, dtype=U8), 2)),
                     ("widen_mxfp4", (x, e, 2, 0)), ("widen_mxfp4", (q, e, 2, 3)), ("widen_mxfp4", (q, e, 3, 0))):
        assert getattr(ext, fn)(*args, 0x77) is None, (fn, args)
    for fn, args in (("dispatch", (x, slots)), ("quant_mxfp4", (x, 2)), ("sort_tokens", (ids, 9))):
        assert getattr(ext, fn)(*args, "stream") is None, fn
        assert getattr(ext, fn)(*args, 0x77) is not None, fn


@pytest.mark.parametrize("i", range(6))
def test_other_threads_run_during_a_call(host, i):
    """The entry point waits (5 s at most) for what another Python thread does."""
    ext, c = host
    x, slots, ids = dev(4, 64, dtype=BF16), dev(4, 3, dtype=I32), dev(4, 3, dtype=I64)
    rows, w, q, e = dev(12, 64, dtype=BF16), dev(4, 3, dtype=F32), dev(4, 32, dtype=U8), dev(4, 2, dtype=E8)
    fn, args = [("sort_tokens", (ids, 9)), ("dispatch", (x, slots)), ("combine", (rows, slots, w, -1)),
                ("combine_grad", (x, rows, slots, w)), ("quant_mxfp4", (x, 2)), ("widen_mxfp4", (q, e, 2, 0))][i]
    stop = threading.Event()

    def opener():
        while not stop.is_set():
            c.rec_gate(1, 1)
            stop.wait(0.002)
    # the gate is shut, then a thread keeps opening it
    c.rec_gate(1, 0)
    thread = threading.Timer(0.05, opener)
    thread.start()
    try:
        assert getattr(ext, fn)(*args, 0x77) is not None
    finally:
        stop.set()
        thread.join()
        c.rec_gate(0, 0)
