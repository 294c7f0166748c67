"""libgmm.so and the compiled binding _moe_ext.so are built and loaded apart:
without the second, the library is still there and every operator still runs
(no GPU; a source of one function stands in for the kernels)."""
import os

import pytest
import torch

from moe_grouped_matrix_amd import _binding, _moe, build
from test_stream_argument import Device, Stream, device


@pytest.fixture
def place(tmp_path, monkeypatch):
    """The build's files in a folder of their own, an old extension among them."""
    src = tmp_path / "one.cpp"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "SOURCES", [str(src)])
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgmm.so"))
    monkeypatch.setattr(build, "EXT", str(tmp_path / "_moe_ext.so"))
    (tmp_path / "_moe_ext.so").write_text("old")
    try:
        build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    return tmp_path


def left(place):
    return sorted(n for n in os.listdir(place) if n != "one.cpp")


def test_the_library_is_built_where_the_extension_cannot_be(place, monkeypatch):
    for command in (["false"], [str(place / "no-such-compiler")]):
        monkeypatch.setattr(build, "_ext_command", lambda out, c=command: c)
        with pytest.warns(UserWarning, match="_moe_ext.so was not built"):
            assert build.build() == str(place / "libgmm.so")
        assert left(place) == ["libgmm.so"]  # nor is the old one left to be loaded

    def no_torch(out):
        raise ImportError("no torch")
    monkeypatch.setattr(build, "_ext_command", no_torch)
    with pytest.warns(UserWarning, match="no torch"):
        build.build()
    monkeypatch.setattr(build, "_ext_command", lambda out: ["cp", str(place / "one.cpp"), out])
    build.build()
    assert left(place) == ["_moe_ext.so", "libgmm.so"]


def test_a_library_that_does_not_compile_changes_nothing(place, monkeypatch):
    (place / "one.cpp").write_text("no c++")
    monkeypatch.setattr(build, "_ext_command", lambda out: ["cp", str(place / "one.cpp"), out])
    with pytest.raises(RuntimeError, match="hipcc failed"):
        build.build()
    assert left(place) == ["_moe_ext.so"] and (place / "_moe_ext.so").read_text() == "old"


@pytest.mark.filterwarnings("error")
@pytest.mark.parametrize("there", [False, True])
def test_operators_run_without_the_extension(tmp_path, monkeypatch, there):
    path = tmp_path / "_moe_ext.so"
    if there:
        path.write_text("not a library")
    ran = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: ran.append(name) or 0

    monkeypatch.setattr(_binding, "_lib", Library())
    monkeypatch.setattr(_binding, "_handles", {0: 1})
    monkeypatch.setattr(_moe, "_ext", None)
    monkeypatch.setattr(_moe, "EXT_PATH", str(path))
    monkeypatch.setattr(_moe, "_current", lambda t: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    x, slots, out = device(6, 64), device(6, 2, dtype=torch.int32), device(12, 64)
    strided = torch.empty_strided
    monkeypatch.setattr(torch, "empty_strided", lambda *a, device=None, **kw: strided(*a, **kw).as_subclass(Device))
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        assert tuple(_moe.dispatch(x, slots).shape) == (12, 64)
    assert _moe.dispatch(x, slots, out=out, stream=Stream(3)) is out  # (no second warning: those are errors here)
    assert ran == ["gmm_dispatch_run"] * 2



def test_threads_load_one_extension(monkeypatch):
    """A second load would forget the handles that the first one was given."""
    import threading
    if not os.path.exists(_moe.EXT_PATH):
        build.build()
    monkeypatch.setattr(_moe, "_ext", None)
    real, loads = _moe.importlib.util.module_from_spec, []
    monkeypatch.setattr(_moe.importlib.util, "module_from_spec", lambda spec: loads.append(spec) or real(spec))
    barrier, got = threading.Barrier(8), []

    def run():
        barrier.wait()
        got.append(_moe._load_ext())
    threads = [threading.Thread(target=run) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(loads) == 1 and len(got) == 8 and all(e is got[0] for e in got)
