"""Checks on the gfx950 code of the 8-bit products (CPU only: hipcc cross-compiles, nothing runs).

The tiled kernel fills LDS with direct loads whose destination is M0, written in the same inline assembly
as the load; no other instruction may name M0.  Its accumulators and fragments have to stay in registers:
a spilled accumulator would cost several times the product.
"""

import re
import shutil

import pytest

from tests.test_codegen import _compile, _hipcc, _kernels, m0_violations


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if _hipcc() is None and shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")
    return _compile(tmp_path_factory.mktemp("fp8"), "fp8_gemm.hip")


def test_m0_is_written_by_the_load_helpers_only(asm):
    kernels = _kernels(asm, "_ZN3nms")
    assert len(kernels) >= 24
    for name, lines in kernels.items():
        assert not m0_violations(lines), name


def test_product_kernels_do_not_spill(asm):
    spills = re.findall(r"\.name:\s+(\S*fp8_gemm\S*)\n(?:.*\n)*?\s+\.vgpr_spill_count:\s+(\d+)", asm)
    assert len(spills) >= 24
    assert all(int(n) == 0 for _, n in spills), [s for s in spills if int(s[1])]


def test_tiled_kernel_waits_before_it_meets(asm):
    """Every barrier of the tiled kernels has the wave's own loads (vmcnt) or LDS operations (lgkmcnt)
    waited for first."""
    for name, lines in _kernels(asm, "_ZN3nms").items():
        if "tile_kernel" not in name:
            continue
        code = [l.split(";")[0].strip() for l in lines]
        code = [c for c in code if c and not c.startswith(".")]
        bars = [i for i, c in enumerate(code) if c == "s_barrier"]
        assert bars, name
        for i in bars:
            assert code[i - 1].startswith("s_waitcnt") and "lgkmcnt(0)" in code[i - 1], (name, code[i - 1])
        assert any(c.startswith("s_waitcnt vmcnt(0)") for c in code), name
