"""Refusals of the 8-bit products' binding for operands of another rank (CPU: the device check is lifted, and
nothing reaches the library)."""

import pytest
import torch

from sparse_matmul_ffns_amd import nmsparse as nm

T8 = torch.float8_e4m3fn


class Library:
    def __getattr__(self, name):
        def reached(*args):
            raise AssertionError("the call reached the library")
        return reached


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setattr(nm, "_dev", lambda *ts: None)
    monkeypatch.setattr(nm, "_stream", lambda: None)
    monkeypatch.setattr(nm, "lib", Library)


def _q(*shape):
    return torch.zeros(*shape, dtype=torch.uint8).view(T8)


@pytest.mark.parametrize("bad", ["A", "sa", "B", "sb", "offsets"])
def test_products_refuse_other_ranks(bad):
    good = dict(A=_q(4, 256), sa=torch.ones(2, 4), B=_q(128, 256), sb=torch.ones(1, 2))
    rows = dict(good, B=_q(3, 128, 256), sb=torch.ones(3, 1, 2), offsets=torch.zeros(4, dtype=torch.int32))
    red = dict(good, sb=torch.ones(2, 128), offsets=torch.zeros(4, dtype=torch.int32))
    for call, args in ((nm.fp8_gemm_nt, good), (nm.fp8_gemm_nt_grouped, rows), (nm.fp8_gemm_nt_grouped_k, red)):
        if bad not in args:
            continue
        for other in (args[bad].reshape(-1).contiguous(), args[bad].reshape(1, 1, *args[bad].shape)):
            if bad == "offsets" and other.dim() == 1:
                other = other[:0]
            with pytest.raises(ValueError):
                call(**dict(args, **{bad: other}))
    with pytest.raises(AssertionError):
        nm.fp8_gemm_nt(**good)


@pytest.mark.parametrize("bad", ["sa", "sb"])
def test_scales_of_one_dimension(bad):
    """As many entries as the scales have rows."""
    args = dict(A=_q(4, 256), sa=torch.ones(2, 4), B=_q(128, 256), sb=torch.ones(2, 128), b_block=1)
    args[bad] = torch.ones(2)
    with pytest.raises(ValueError):
        nm.fp8_gemm_nt(**args)
