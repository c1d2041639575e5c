"""The work memory that the binding asks for by the operands' strides and addresses (CPU)."""

import pytest
import torch

from sparse_matmul_ffns_amd import nmsparse as nm


def _matrix(R, C, ld, off=0):
    return torch.zeros(off + (R - 1) * ld + C, dtype=torch.bfloat16)[off:].as_strided((R, C), (ld, 1))


@pytest.fixture
def asked(monkeypatch):
    seen = []

    def need(call, M, N, K, aligned):
        seen.append(aligned)
        return 0

    class Library:
        def __getattr__(self, name):
            return lambda *args: 0
    monkeypatch.setattr(nm, "_linear_work_bytes", need)
    monkeypatch.setattr(nm, "_here", lambda *ts: None)
    monkeypatch.setattr(nm, "_stream", lambda: None)
    monkeypatch.setattr(nm, "lib", Library)
    return seen


@pytest.mark.parametrize("ld,off,want", [(16, 0, True), (24, 0, True), (20, 0, False), (16, 1, False), ((1 << 22) - 8, 0, True), (1 << 22, 0, False),
                                         ((1 << 22) + 8, 0, False)])
def test_aligned(asked, ld, off, want):
    a, b = _matrix(3, 16, ld, off), _matrix(16, 16, 16)
    nm.linear_fwd(a, b), nm.linear_fwd(b, _matrix(3, 16, ld, off))
    nm.linear_bwd_x(a, b), nm.linear_bwd_x(_matrix(3, 3, 8), a)
    nm.linear_bwd_w(a, _matrix(3, 16, 16)), nm.linear_bwd_w(_matrix(3, 16, 16), a)
    assert asked == [want] * 6
