"""The schedule of the large-group kernel for microscaled fp4 weights
(gmm_mxw_big.hpp), on the CPU.

Its K loop waits on constant vmcnt values.  A wave's memory operations complete
in issue order, and `s_waitcnt vmcnt(n)` returns once at most n are
outstanding; so a wait for a stage is good when the stage's last load has at
least n operations behind it, and idle-free when it has exactly n.  The first
test replays a wave's issue order and checks every wait and every reuse of a
stage; the second compiles the kernel and checks that the compiler kept every
operation that the constants count."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_grouped_matrix_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
S, OPS = 3, 6


def _replay(KT, tiles, E):
    """(wait, operations behind the awaited stage's last load) for every
    middle of a step, checking that a stage is loaded only when the step that
    used it lies behind a barrier."""
    issued, waits, holds = [], [], {}

    def load(tile, k, slot):
        issued.extend([("L", tile, k)] * (OPS + (1 if k == 0 and tile else 0)))
        holds[slot] = (tile, k)

    load(0, 0, 0)
    load(0, 1, 1)
    waits.append((0, 0))
    slot = 0
    for t in range(tiles):
        for k in range(KT):
            assert holds[slot] == (t, k)
            need = (t, k + 1) if k + 1 < KT else (t + 1, 0)
            last = max((i for i, op in enumerate(issued) if op == ("L",) + need), default=None)
            assert last is not None and holds[(slot + 1) % S] == need
            waits.append((E if k == 0 and t else 0 if t else 0, len(issued) - 1 - last))
            before = (slot + S - 1) % S
            if t or k:
                # the step before this one used it, and every wave is past that step
                assert holds[before] == ((t, k - 1) if k else (t - 1, KT - 1))
            nk = k + 2
            load(*((t, nk) if nk < KT else (t + 1, nk - KT)), before)
            if k == KT - 1:
                issued.extend([("E", t)] * E)
            slot = (slot + 1) % S
    return waits


@pytest.mark.parametrize("E", [16, 32])
@pytest.mark.parametrize("KT", [3, 4, 5, 11, 22])
def test_waits_are_exact(KT, E):
    for n, behind in _replay(KT, 4, E):
        assert n == behind


def test_a_shorter_ring_is_caught():
    """The replay is not vacuous: a wait that allows the E stores at a tile's
    second step as well would let a stage's loads be outstanding."""
    waits = _replay(5, 3, 16)
    assert any(behind == 0 and n == 0 for n, behind in waits[1:])
    assert all(16 > behind for n, behind in waits if n == 0)


def test_the_compiler_kept_every_counted_operation(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from moe_grouped_matrix_amd import build
    out = tmp_path / "mxw.s"
    flags = [f for f in build.HIPCC_FLAGS if f != "-fPIC"] + build.EXTRA_FLAGS.get("gmm_mxw.hip", [])
    res = subprocess.run([HIPCC] + flags + ["-I" + os.path.join(ROOT, "include"), "-S", "--cuda-device-only",
                                            os.path.join(CSRC, "gmm_mxw.hip"), "-o", str(out)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    asm = out.read_text()
    seen = 0
    for name in re.findall(r"^(_ZN4gmmk18gmm_mxw_big_kernel\S*):", asm, re.M):
        body = asm[asm.index(name + ":"):]
        lines = [ln.strip() for ln in body[:body.index(".Lfunc_end")].split("\n")]
        stores = 32 if "MxwBigCfgILb1E" in name else 16
        # a full and a half tile's epilogue
        assert sum(ln.startswith("buffer_store") for ln in lines) == 2 * stores, name
        # the prologue's two stages, and four steps (first, middle, next tile's
        # first and second loads) of a full and of a half tile
        lds = [ln for ln in lines if ln.startswith("buffer_load") and ln.endswith("lds")]
        assert sum("dwordx4" in ln for ln in lds) == 5 * (2 + 8), name
        assert sum("dwordx4" not in ln for ln in lds) == 2 + 8 + 1 + 2, name  # scales; bias rows
        # a step's products: 4 x 4 x 2 of a full tile, half of them of a half one
        assert sum("v_mfma_f32_32x32x16_bf16" in ln for ln in lines) == 4 * (32 + 16), name
        seen += 1
    assert seen == 4  # bf16 / f32 output, with / without bias
