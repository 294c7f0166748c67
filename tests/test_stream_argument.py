"""What the binding does with memory when a call runs on a stream of the
caller's choice (stream=), on the CPU: outputs that it makes are allocated on
that stream, and every tensor of the call is kept from reuse until the stream
is done with it.  The library and the device allocator are stood in for by
Python objects that keep account."""
import contextlib
import ctypes

import pytest
import torch

from moe_grouped_matrix_amd import _binding, _moe

DEV = torch.device("cuda", 0)
_empty, _empty_strided = torch.empty, torch.empty_strided


class Device(torch.Tensor):
    """A host tensor that passes for a device tensor; the streams that its
    memory is kept for are noted by storage (a view keeps the whole)."""
    is_cuda = True
    device = DEV
    kept = {}

    def record_stream(self, stream):
        self.kept.setdefault(self.untyped_storage().data_ptr(), []).append(stream)


def kept(t):
    return Device.kept.get(t.untyped_storage().data_ptr(), [])


def device(*shape, dtype=torch.bfloat16):
    return _empty(shape, dtype=dtype).as_subclass(Device)


class Stream:
    device = DEV

    def __init__(self, number):
        self.cuda_stream = number


class Library:
    """Every entry point queues nothing and says that all is well."""

    def __init__(self):
        self.raw = []

    def __getattr__(self, name):
        def call(*args):
            last = args[-1]
            self.raw.append(last.value if isinstance(last, ctypes.c_void_p) else last)
            return 0
        return call


class Ext:
    def set_handle(self, *_):
        pass


@pytest.fixture
def streams(monkeypatch):
    """(the caller's current stream, another one, the library)"""
    current, other = Stream(0x10), Stream(0x20)
    now = [current]

    @contextlib.contextmanager
    def use(stream):
        now.append(stream if stream is not None else now[-1])
        yield
        now.pop()

    def made(real):
        def make(*args, device=None, **kw):
            t = real(*args, **kw).as_subclass(Device)
            t.made_on = now[-1]
            return t
        return make

    lib = Library()
    monkeypatch.setattr(Device, "kept", {})
    monkeypatch.setattr(torch, "empty", made(_empty))
    monkeypatch.setattr(torch, "empty_strided", made(_empty_strided))
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now[-1])
    monkeypatch.setattr(_binding, "_lib", lib)
    monkeypatch.setattr(_binding, "_handles", {0: 1})
    monkeypatch.setattr(_moe, "_ext", Ext())
    return current, other, lib


def check(streams, call, inputs, given=()):
    """call(stream) gives the outputs, the caller's own (`given`) among them."""
    current, other, lib = streams
    outs = call(other)
    outs = outs if isinstance(outs, tuple) else (outs,)
    assert lib.raw[-1] == other.cuda_stream
    for t in inputs:
        assert other in kept(t), "an input may be reused while the stream reads it"
    for t in outs:
        if any(t is g for g in given):
            assert other in kept(t), "the caller's output may be reused while the stream writes it"
        else:
            assert t.made_on is other, "an output was allocated on another stream than the one that writes it"
            assert current in kept(t), "an output may be reused while the caller's stream reads it"
    for g in given:
        assert any(g is t for t in outs)


def products():
    lhs, rhs, sizes = device(8, 64), device(2, 16, 64), device(2, dtype=torch.int32)
    scale, bias, lscale = device(2, 1, 1, 16, dtype=torch.float32), device(2, 1, 16), device(8, 1, dtype=torch.float32)
    return lhs, rhs, sizes, scale, bias, lscale


def test_gmm(streams):
    lhs, rhs, sizes, scale, bias, lscale = ins = products()
    check(streams, lambda st: _binding.gmm(lhs, rhs, sizes, rhs_scale=scale, rhs_bias=bias, lhs_scale=lscale, stream=st),
          ins)


def test_gmm_with_outputs_and_an_offset(streams):
    ins = products()
    out, keep, off = device(8, 16), device(8, 16), device(1, dtype=torch.int32)
    check(streams, lambda st: _binding.gmm(*ins[:3], out=out, existing_out=keep, group_offset=off, stream=st),
          ins[:3] + (keep, off), (out,))
    ins, into = products(), device(8, 16)
    check(streams, lambda st: _binding.gmm(*ins[:3], existing_out=into, stream=st), ins[:3], (into,))


def test_a_misaligned_offset_is_copied_on_the_stream(streams):
    ins = products()
    odd = device(5, dtype=torch.int32)[1:2]
    assert odd.data_ptr() % 16
    clones = []
    Device.clone = lambda self: clones.append(torch.cuda.current_stream()) or torch.Tensor.clone(self)
    try:
        check(streams, lambda st: _binding.gmm(*ins[:3], group_offset=odd, stream=st), ins[:3])
    finally:
        del Device.clone
    assert clones == [streams[1]]


def test_gmm_of_packed_weights(streams):
    lhs, sizes = device(8, 64), device(2, dtype=torch.int32)
    q, scale = device(2, 16, 32, dtype=torch.uint8), device(2, 2, 1, 16, dtype=torch.float8_e8m0fnu)
    check(streams, lambda st: _binding.gmm(lhs, q, sizes, rhs_scale=scale, rhs_format="fp4_e2m1", stream=st),
          (lhs, q, sizes, scale))


@pytest.mark.parametrize("no_alloc", [False, True])
def test_tgmm(streams, no_alloc):
    lhs, rhs, sizes = device(8, 64), device(8, 16), device(2, dtype=torch.int32)
    check(streams, lambda st: _binding.tgmm(lhs, rhs, sizes, no_alloc=no_alloc, stream=st), (lhs, rhs, sizes))
    lhs, rhs, sizes, out = device(8, 64), device(8, 16), device(2, dtype=torch.int32), device(2, 64, 16)
    check(streams, lambda st: _binding.tgmm(lhs, rhs, sizes, out=out, no_alloc=no_alloc, stream=st), (lhs, rhs, sizes),
          (out,))


def test_quant_fp8_and_widen_scales(streams):
    x = device(8, 128)
    check(streams, lambda st: _binding.quant_fp8(x, stream=st), (x,))
    x, q, s = device(8, 128), device(8, 128, dtype=torch.float8_e4m3fn), device(8, 1, dtype=torch.float32)
    check(streams, lambda st: _binding.quant_fp8(x, q=q, scale=s, stream=st), (x,), (q, s))
    src = device(3, 4, dtype=torch.float8_e8m0fnu)
    check(streams, lambda st: _binding.widen_scales(src, stream=st), (src,))
    src, out = device(3, 4, dtype=torch.float8_e8m0fnu), device(3, 4, dtype=torch.float32)
    check(streams, lambda st: _binding.widen_scales(src, out=out, stream=st), (src,), (out,))


def test_a_stream_of_another_device_is_refused(streams):
    far = Stream(0x30)
    far.device = torch.device("cuda", 1)
    ins = products()
    for call in (lambda: _binding.gmm(*ins[:3], stream=far), lambda: _binding.tgmm(ins[0], ins[0], ins[2], stream=far),
                 lambda: _binding.quant_fp8(device(8, 128), stream=far),
                 lambda: _binding.widen_scales(device(3, dtype=torch.float32), stream=far),
                 lambda: _moe.dispatch(ins[0], device(8, 1, dtype=torch.int32), stream=far)):
        with pytest.raises(_binding.GmmInvalid, match="stream is on"):
            call()
    assert streams[2].raw == []


def moe_calls():
    """(name, call(stream, **given), inputs, {name of an output: the caller's}) of the token and fp4 operators."""
    i32, f32, e8 = torch.int32, torch.float32, torch.float8_e8m0fnu
    ids, slots, x = device(6, 2, dtype=torch.int64), device(6, 2, dtype=i32), device(6, 64)
    rows, w = device(12, 64), device(6, 2, dtype=f32)
    q, e = device(6, 32, dtype=torch.uint8), device(6, 2, dtype=e8)
    return [
        ("sort_tokens", lambda **kw: _moe.sort_tokens(ids, 4, **kw), (ids,),
         dict(group_sizes=device(4, dtype=i32), slot_row=device(6, 2, dtype=i32))),
        ("dispatch", lambda **kw: _moe.dispatch(x, slots, **kw), (x, slots), dict(out=device(12, 64))),
        ("combine", lambda **kw: _moe.combine(rows, slots, w, **kw), (rows, slots, w), dict(out=device(6, 64))),
        ("combine_grad", lambda **kw: _moe.combine_grad(x, rows, slots, w, **kw), (x, rows, slots, w),
         dict(drows=device(12, 64), dweights=device(6, 2, dtype=f32))),
        ("quant_mxfp4", lambda **kw: _moe.quant_mxfp4(x, **kw), (x,),
         dict(q=device(6, 32, dtype=torch.uint8), scale=device(6, 2, dtype=e8))),
        ("widen_mxfp4", lambda **kw: _moe.widen_mxfp4(q, e, **kw), (q, e), dict(out=device(6, 64))),
    ]


@pytest.mark.parametrize("i", range(6))
def test_token_and_fp4_operators(streams, i):
    name, call, ins, _ = moe_calls()[i]
    check(streams, lambda st: call(stream=st), ins)
    name, call, ins, given = moe_calls()[i]
    check(streams, lambda st: call(stream=st, **given), ins, tuple(given.values()))
    name, call, ins, given = moe_calls()[i]
    first = dict(list(given.items())[:1])
    check(streams, lambda st: call(stream=st, **first), ins, tuple(first.values()))
