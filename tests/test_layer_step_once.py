"""A step reads what it writes, so a call of adamw() asks the library for it
once: a HIP error, after which a part of it may have been queued, is raised and
not tried again the long way (csrc/moe_ext.cpp bound to an entry point that
counts its calls and returns a chosen status; host tensors pass for tensors of
device 0)."""
import ctypes
import importlib.util
import os
import subprocess

import pytest
import torch

from moe_grouped_matrix_amd import _binding, _layer, _moe, build
from test_layer_ext_host import ENTRIES, SOURCE
from test_moe_ext_host import dev

TAKE = """  g_args = *a;
  return take({}, {(double)(uintptr_t)st});
"""
COUNTED = """  g_args = *a;
  ++g_calls;
  return (gmm_status)g_status;
"""
KNOBS = """
static int g_calls, g_status;
extern "C" void rec_expect(int status) { g_calls = 0; g_status = status; }
extern "C" int rec_calls() { return g_calls; }
"""
OK, INVALID, UNSUPPORTED, HIP = 0, _binding.GMM_E_INVALID, _binding.GMM_E_UNSUPPORTED, _binding.GMM_E_HIP


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("ext")
    assert TAKE in SOURCE
    source = SOURCE.replace(TAKE, COUNTED).replace('static gmm_tensor g_taken', KNOBS + 'static gmm_tensor g_taken', 1)
    (d / "t.cpp").write_text(source)
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


@pytest.fixture
def step(host, monkeypatch):
    """step(status) -> how often the step was asked for, and what adamw() raised"""
    ext, c = host
    long_way = []

    class Library:
        def gmm_adamw_run(self, *args):
            long_way.append(args)
            return c.status

        def gmm_last_error(self, h):
            return b"a text"

    monkeypatch.setattr(_binding, "_lib", Library())
    monkeypatch.setattr(_binding, "_handles", {0: 1, None: 1})
    monkeypatch.setattr(_layer, "_current", lambda t: 0x77)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x77, raising=False)
    monkeypatch.setattr(_moe, "_ext", ext)

    def run(status, forms=list):
        c.status = status
        c.rec_expect(status)
        long_way.clear()
        col = lambda d: forms([dev(600, dtype=d) for _ in range(3)])  # noqa: E731
        raised = None
        try:
            _layer.adamw(col(torch.float32), col(torch.bfloat16), col(torch.float32), col(torch.float32), 1, lr=0.1)
        except _binding.GmmError as e:
            raised = e
        return c.rec_calls(), len(long_way), raised
    return run


def test_done_at_once(step):
    assert step(OK) == (1, 0, None)


def test_a_failed_step_is_not_asked_for_again(step):
    short, long_way, raised = step(HIP)
    assert (short, long_way) == (1, 0)
    assert type(raised) is _binding.GmmError and raised.status == HIP and "a text" in str(raised)


@pytest.mark.parametrize("status,cls", [(INVALID, _binding.GmmInvalid), (UNSUPPORTED, _binding.GmmUnsupported)])
def test_a_refused_step_is_told_why(step, status, cls):
    """(nothing was queued: the long way meets the same refusal)"""
    short, long_way, raised = step(status)
    assert (short, long_way) == (1, 1) and type(raised) is cls


def test_the_long_way_asks_once_too(step):
    for status in (OK, HIP):
        short, long_way, raised = step(status, _Sequence)
        assert (short, long_way) == (0, 1) and (raised is None) == (status == OK)


class _Sequence:
    """Neither a list nor a tuple: the compiled code does not take it."""

    def __init__(self, ts):
        self.ts = ts

    def __len__(self):
        return len(self.ts)

    def __getitem__(self, i):
        return self.ts[i]


def test_what_the_extension_returns(host):
    ext, c = host
    args = [[dev(8, dtype=torch.float32)] for _ in range(4)] + [None, None, None, 1, 0.1, 0.9, 0.99, 1e-8, 0.0, None, 0x77]
    for status, want in ((OK, True), (INVALID, None), (UNSUPPORTED, None), (HIP, HIP), (99, 99)):
        c.rec_expect(status)
        got = ext.adamw(*args)
        assert got == want and type(got) is type(want) and c.rec_calls() == 1
