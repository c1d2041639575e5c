"""Waits of the tiled 8-bit products' direct-to-LDS loads in the compiled gfx950 code (CPU only).

A wave's loads into LDS are seen by the other waves only if the wave has waited for them (vmcnt 0) before
the barrier that publishes the stage, and none may land after the workgroup has ended.  Both are checked
along every path of each kernel's control-flow graph: no load of LDS is in flight at a barrier or at the
end.  A copy of the source without the wait must fail the check.
"""

import os
import re
import shutil

import pytest

from tests import test_codegen as cg


def in_flight(asm_lines):
    """(line, instruction) of the barriers and ends that a path reaches with a load of LDS in flight; the
    number of such loads and of barriers in the kernel."""
    blocks = cg._blocks(asm_lines)
    bad, seen, work, loads, bars = set(), set(), [(0, False)], set(), set()
    while work:
        k, fly = work.pop()
        if (k, fly) in seen:
            continue
        seen.add((k, fly))
        for i, c, _ in blocks[k]["insns"]:
            if c.startswith("global_load_lds_") or (c.startswith("buffer_load_") and re.search(r"\blds\b", c)):
                loads.add(i)
                fly = True
            elif c.startswith("s_waitcnt") and "vmcnt(0)" in c:
                fly = False
            elif c == "s_barrier" or c.startswith("s_endpgm"):
                if c == "s_barrier":
                    bars.add(i)
                if fly:
                    bad.add((i + 1, c))
        work += [(s, fly) for s in blocks[k]["succ"]]
    return sorted(bad), len(loads), len(bars)


def _tiled(asm):
    out = {n: b for n, b in cg._kernels(asm, "_ZN3nms").items() if "fp8_gemm_tile_kernel" in n}
    assert len(out) >= 16
    return out


@pytest.mark.skipif(cg._hipcc() is None, reason="hipcc not available")
def test_no_load_is_in_flight_at_a_barrier_or_at_the_end(tmp_path):
    for name, lines in _tiled(cg._compile(tmp_path, "fp8_gemm.hip")).items():
        bad, loads, bars = in_flight(lines)
        assert loads >= 18 and bars >= 4, name     # two stages of eight loads and the scales; land()s of both kinds
        assert not bad, (name, bad[:5])


@pytest.mark.skipif(cg._hipcc() is None, reason="hipcc not available")
@pytest.mark.parametrize("old,new", [("    wait_vmcnt<0>();\n    lds_barrier();", "    lds_barrier();"),
                                     ("    wait_vmcnt<0>();   // no load may land", "    // no load may land")])
def test_a_missing_wait_is_found(tmp_path, monkeypatch, old, new):
    src = tmp_path / "csrc"
    shutil.copytree(cg.CSRC, src)
    text = (src / "fp8_gemm.hip").read_text()
    assert text.count(old) == 1
    (src / "fp8_gemm.hip").write_text(text.replace(old, new))
    monkeypatch.setattr(cg, "CSRC", os.fspath(src))
    found = [bool(in_flight(lines)[0]) for lines in _tiled(cg._compile(tmp_path, "fp8_gemm.hip")).values()]
    assert all(found)


def test_the_check_follows_paths():
    load, wait, bar, end = "\tbuffer_load_dwordx4 v0, s[0:3], 0 offen lds", "\ts_waitcnt vmcnt(0)", "\ts_barrier", "\ts_endpgm"
    assert not in_flight([load, wait, bar, end])[0]
    assert in_flight([load, bar, wait, end])[0] == [(2, "s_barrier")]
    assert in_flight([load, "\ts_waitcnt vmcnt(1)", bar, wait, end])[0]
    assert in_flight([wait, bar, load, end])[0] == [(4, "s_endpgm")]
    # the wait is on one of two paths
    assert in_flight([load, "\ts_cbranch_scc0 .LBB0_2", wait, ".LBB0_2:", bar, wait, end])[0]
    # round a loop
    assert in_flight([".LBB0_1:", bar, load, "\ts_cbranch_scc0 .LBB0_1", wait, end])[0] == [(2, "s_barrier")]
