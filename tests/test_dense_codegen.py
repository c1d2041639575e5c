"""Checks on the gfx950 code of the dense products (CPU only: hipcc cross-compiles, nothing runs).

The tiled kernels fill LDS with direct loads whose destination is M0, written in the same inline assembly as the load;
no other instruction may name M0.  Accumulators and fragments have to stay in registers.  No load may land in LDS after
the epilogue has begun to use it, or after the workgroup has ended.  And no 16-byte store may have a scalar offset: the compiler
takes such a store's data as read at once and may overwrite its registers in the next instruction, but on the
GPU the last lanes then store what that wrote (seen as wrong values in ragged products).
"""

import re
import shutil

import pytest

from tests import test_codegen as cg

pytestmark = pytest.mark.skipif(cg._hipcc() is None and shutil.which("hipcc") is None, reason="hipcc not available")
SOURCES = ["linear.hip", "linear_act.hip", "norm.hip", "grads.hip", "partials.hip"]


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    return {s: cg._compile(tmp_path_factory.mktemp("dense"), s) for s in SOURCES}


# by tile: the loads of a unit of 64 k in a wave, and what may be in flight at the barrier before the loop and at the one inside it
WAITS = {"LinCfgILi8ELi8E": (16, (16, 8)), "LinCfgILi8ELi4E": (12, (24, 16)), "LinCfgILi4ELi4E": (8, (24, 20))}


def _tiled(text):
    out = {n: b for n, b in cg._kernels(text, "_ZN3nms").items() if "linear_tile_kernel" in n}
    assert len(out) >= 18
    return out


def _code(lines):
    out = [l.split(";")[0].strip() for l in lines]
    return [c for c in out if c and not c.startswith(".")]


def test_m0_is_written_by_the_load_helpers_only(asm):
    for name, lines in _tiled(asm["linear.hip"]).items():
        assert not cg.m0_violations(lines), name


@pytest.mark.parametrize("source", SOURCES)
def test_nothing_spills(asm, source):
    spills = re.findall(r"\.name:\s+(\S+)\n(?:.*\n)*?\s+\.vgpr_spill_count:\s+(\d+)", asm[source])
    assert spills and all(int(n) == 0 for _, n in spills), [s for s in spills if int(s[1])]
    assert "scratch_store" not in asm[source] and "scratch_load" not in asm[source]


@pytest.mark.parametrize("source", SOURCES)
def test_wide_stores_have_no_scalar_offset(asm, source):
    for line in _code(asm[source].splitlines()):
        if re.match(r"buffer_store_dwordx[34]\b", line):
            assert re.search(r"\],\s*0 offen", line), line


def test_loads_are_waited_for(asm):
    """At every barrier of the tiled kernels the wave has waited for its LDS operations and for all but its last steps'
    loads; behind the last of them (the epilogue) for all loads."""
    for name, lines in _tiled(asm["linear.hip"]).items():
        code = _code(lines)
        loads, allowed = next(v for k, v in WAITS.items() if k in name)
        bars = [i for i, c in enumerate(code) if c == "s_barrier"]
        assert len(bars) >= 4, name
        seen = set()
        last = 0
        for i in bars:
            assert "lgkmcnt(0)" in code[i - 1], (name, code[i - 1])
            waits = [re.search(r"vmcnt\((\d+)\)", c) for c in code[max(0, i - 60):i] if c.startswith("s_waitcnt")]
            counts = [int(w.group(1)) for w in waits if w]
            assert counts and min(counts) in (0, *allowed), (name, counts)
            last = i if min(counts) == 0 else last
            seen.add(min(counts))
        assert seen == {0, *allowed}, (name, seen)
        dma = [i for i, c in enumerate(code) if c.startswith("buffer_load_") and re.search(r"\blds\b", c)]
        assert len(dma) >= 4 * loads, name
        ends = _in_flight_at_the_end(lines)
        assert not ends, (name, ends)


def _in_flight_at_the_end(lines):
    blocks = cg._blocks(lines)
    seen, work, bad = set(), [(0, False)], set()
    while work:
        k, fly = work.pop()
        if (k, fly) in seen:
            continue
        seen.add((k, fly))
        for i, c, _ in blocks[k]["insns"]:
            if c.startswith("buffer_load_") and re.search(r"\blds\b", c):
                fly = True
            elif c.startswith("s_waitcnt") and "vmcnt(0)" in c:
                fly = False
            elif c.startswith("s_endpgm") and fly or c.startswith("ds_write") and fly:
                bad.add((i + 1, c))
        work += [(s, fly) for s in blocks[k]["succ"]]
    return sorted(bad)


def test_the_check_finds_a_missing_wait():
    load, wait, end = "\tbuffer_load_dwordx4 v0, s[0:3], 0 offen lds", "\ts_waitcnt vmcnt(0)", "\ts_endpgm"
    assert not _in_flight_at_the_end([load, wait, end])
    assert _in_flight_at_the_end([load, "\ts_waitcnt vmcnt(8)", end])
    assert _in_flight_at_the_end([load, "\tds_write_b128 v0, v[0:3]", wait, end])
