"""The waits of the large-group kernel for microscaled fp4 weights, read out of
its source (gmm_mxw_big.hpp) and replayed on the CPU.

A wave's memory operations complete in issue order, and `s_waitcnt vmcnt(n)`
returns once at most n are outstanding.  The schedule -- ring size, operations a
step, the wait, target and source step of every kstep call of a tile, the
stages' rotation -- is parsed from the kernel, so a changed wait is replayed as
it stands; what the parser does not know fails.  A stage counts as readable only
when the wait before its first read has covered all its loads, and as free only
when the step that read it lies behind a barrier.  The negative tests change the
source text and have to be rejected."""
import os
import re
import subprocess

import pytest

from test_mxw_schedule import CSRC, HIPCC, ROOT

SOURCE = open(os.path.join(CSRC, "gmm_mxw_big.hpp")).read()


class Schedule:
    """What the kernel's text says."""

    def __init__(self, text, out_f32):
        text = re.sub(r"//[^\n]*", "", text)
        self.text = text

        def one(pattern, where=text):
            found = re.findall(pattern, where)
            assert len(found) == 1, (pattern, found)
            return found[0]

        self.S = int(one(r"static constexpr int S = (\d+);"))
        self.OPS = int(one(r"static constexpr int OPS = (\d+);"))
        fm, fn = map(int, one(r"static constexpr int FM = (\d+), FN = (\d+);"))
        st32, st16 = map(int, one(r"static constexpr int ST_BLOCK = OUT_F32 \? (\d+) : (\d+);"))
        one(r"static constexpr int E_FULL = FM \* FN \* ST_BLOCK, E = E_FULL;")
        self.E = fm * fn * (st32 if out_f32 else st16)
        waits = {"WE": self.E, "W0": 0}
        one(r"using WE = std::integral_constant<int, C::E>;")
        one(r"using W0 = std::integral_constant<int, 0>;")

        # the prologue: a bias piece, the first stages in order, then everything waited for
        pro = text[text.index("BigItem cur = decode_big"):text.index("const int swz_r")]
        self.ahead = int(one(r"for \(int s = 0; s < (\d+); \+\+s\)", pro))
        assert len(re.findall(r"mxw_op<C, [0-5]>\(dcur, off, s, N, st, ", pro)) == self.OPS
        one(r"wait_vmcnt<0>\(\);\s*__syncthreads\(\);", pro)

        # a step: wait and barrier before the loads and before the next stage's first read
        step = text[text.index("auto kstep ="):text.index("using T_ = std::true_type")]
        nxt, back = one(r"const int s1 = (.+?), s2 = (.+?);", step)
        names = {"C::S": str(self.S)}

        def turn(expr):
            for k, v in names.items():
                expr = expr.replace(k, v)
            cond, yes, no = re.fullmatch(r"stage == (.+?) \? (.+?) : (.+)", expr).groups()
            return lambda stage: eval(yes if stage == eval(cond) else no, {"stage": stage})
        self.next, self.back = turn(nxt), turn(back)
        one(r"if \(h == 2\) \{\s*wait_vmcnt<WAIT>\(\);", step)
        assert step.index("wait_vmcnt<WAIT>") < step.index("ring_barrier()") < step.index("read_w(st1")
        one(r"if \(h >= 2\) op\(", step)
        one(r"h < 2 \? a_frag\(st, cur, fm, h \+ 2\) : a_frag\(st1, it1, fm, h - 2\)", step)
        assert sorted(re.findall(r"mxw_op<C, (\d)>\(d, off, kd, N, st2, ", step)) == [str(i) for i in range(self.OPS + 1)]
        one(r"stage = s1;", step)

        # a tile: the kstep calls in order, one of them a loop over kt
        tile = text[text.index("auto ktile ="):text.index("const int last = stage")]
        calls = re.findall(r"(for \(int kt = 1; kt \+ 2 < KT; \+\+kt\) )?kstep\(full_tag, (\w+)\{\}, ([TF])_\{\}, "
                           r"([TF])_\{\}, ([TF])_\{\}, ([^)]+)\);", tile)
        assert len(calls) == tile.count("kstep(") and [bool(c[0]) for c in calls] == [False, True, False, False]
        self.calls = [(bool(loop), waits[w], n == "T", b == "T", last == "T", kd) for loop, w, n, b, last, kd in calls]
        one(r"big_epilogue<C, FMA, C::BIAS>", text)

    def steps(self, KT):
        """(wait, loads for the next tile, with the bias piece, last, step loaded) of a tile's steps."""
        out = []
        for loop, wait, nxt, bias, last, kd in self.calls:
            for kt in range(1, KT - 2) if loop else (0,):
                out.append((wait, nxt, bias, last, eval(kd, {"kt": kt})))
        return out


def replay(s, KT, tiles):
    """Every wait as (allowed, operations behind the last load that it is for); asserts where a stage is read
    before its loads are known to be complete, or loaded while it may still be read."""
    issued, done, slots = [], 0, [None] * s.S

    def load(tile, k, slot, bias):
        for _ in range(s.OPS + bias):
            issued.append(("load", tile, k))
        slots[slot] = (tile, k)

    def readable(tile, k):
        last = max(i for i, op in enumerate(issued) if op == ("load", tile, k))
        return last < done

    for k in range(s.ahead):
        load(0, k, k, k == 0)
    done = len(issued)
    stage, exact = 0, []
    for t in range(tiles):
        steps = s.steps(KT)
        assert len(steps) == KT, "a tile takes another number of steps"
        for k, (wait, nxt, bias, last, kd) in enumerate(steps):
            assert last == (k == KT - 1)
            assert slots[stage] == (t, k), "the stage holds another step"
            assert readable(t, k), "the step's stage is read before it is complete"
            need = (t, k + 1) if k + 1 < KT else (t + 1, 0)
            at = max((i for i, op in enumerate(issued) if op == ("load",) + need), default=None)
            assert at is not None and slots[s.next(stage)] == need, "the next stage is not on its way"
            exact.append((wait, len(issued) - 1 - at if at >= done else None))
            done = max(done, len(issued) - wait)
            assert readable(*need), f"tile {t} step {k}: vmcnt({wait}) lets the next stage be read before it is complete"
            # past the barrier every wave is past the step before this one
            free = s.back(stage)
            assert slots[free] is None or slots[free] == ((t, k - 1) if k else (t - 1, KT - 1)), \
                "a stage is loaded over while it may still be read"
            load(t + 1 if nxt else t, kd, free, bias)
            if last:
                issued.extend([("store", t)] * s.E)
            stage = s.next(stage)
    return exact


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("KT", [3, 4, 5, 11, 22, 65])
def test_every_stage_is_complete_before_it_is_read(KT, out_f32):
    for wait, behind in replay(Schedule(SOURCE, out_f32), KT, 5):
        # and no wait holds up a newer operation
        assert behind is None or wait == behind


def changed(old, new, count=1):
    assert SOURCE.count(old) == count, (old, SOURCE.count(old))
    return SOURCE.replace(old, new)


STEADY = "kstep(full_tag, W0{}, F_{}, F_{}, F_{}, kt + 2);"
NEXT0 = "kstep(full_tag, W0{}, T_{}, T_{}, F_{}, 0);"
NEXT1 = "kstep(full_tag, W0{}, T_{}, F_{}, T_{}, 1);"
BROKEN = {
    "stores allowed in the steady steps": changed(STEADY, STEADY.replace("W0", "WE")),
    "stores allowed in the step before the last": changed(NEXT0, NEXT0.replace("W0", "WE")),
    "stores allowed in the last step": changed(NEXT1, NEXT1.replace("W0", "WE")),
    "more stores allowed than there are": changed("std::integral_constant<int, C::E>", "std::integral_constant<int, C::E + 1>"),
    "a ring of two stages": changed("static constexpr int S = 3;", "static constexpr int S = 2;"),
    "loads into the stage that is read next": changed(
        "s2 = stage == 0 ? C::S - 1 : stage - 1;", "s2 = stage == C::S - 1 ? 0 : stage + 1;"),
    "loads into the stage that is being read": changed(
        "s2 = stage == 0 ? C::S - 1 : stage - 1;", "s2 = stage == 0 ? stage : stage;"),
    "the wait after the read": changed("if (h == 2) {\n        wait_vmcnt<WAIT>();", "if (h == 3) {\n        wait_vmcnt<WAIT>();"),
    "a step too few in flight": changed("for (int s = 0; s < 2; ++s)", "for (int s = 0; s < 1; ++s)"),
    "the wrong step of the next tile": changed(NEXT1, NEXT1.replace("1);", "2);")),
    "a step left out": changed("kt + 2 < KT", "kt + 3 < KT"),
}


@pytest.mark.parametrize("what", sorted(BROKEN))
def test_a_broken_schedule_is_rejected(what):
    with pytest.raises(AssertionError):
        for KT in (3, 5):
            replay(Schedule(BROKEN[what], False), KT, 4)


def test_spilled_registers_stay_out_of_the_steady_steps(tmp_path):
    """Scratch accesses would be counted by the steps' waits: the compiled loops
    over a tile's steady steps hold none, in any variant."""
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
    names = re.findall(r"^(_ZN4gmmk18gmm_mxw_big_kernel\S*):", asm, re.M)
    assert len(names) == 4
    for name in names:
        body = asm[asm.index(name + ":"):]
        blocks = re.split(r"^(?=\.LBB)", body[:body.index(".Lfunc_end")], flags=re.M)
        loops = [b for b in blocks if re.search(r"Inner Loop Header: Depth=2", b) and "v_mfma" in b]
        assert sorted(b.count("v_mfma") for b in loops) == [16, 32], name  # a half and a full tile's
        for b in loops:
            assert "scratch_" not in b, name
