"""The norm's gradient where a workgroup takes many rows (GPU): random rows everywhere, for every number of threads.

Tolerances as in tests/test_gpu_dense.py (U = 2^-24): a row's mean is off by 70 U of the mean of |g xh|; dw adds a row's terms in chains of
T / groups + 1, then over at most 4 waves and 512 groups (16 waves of 32 steps)."""

import numpy as np
import pytest
import torch

import sparse_matmul_ffns_amd as nm
from oracle import dense_oracle as O
from tests.gpu_util import require_gpu
from tests.test_gpu_dense import U, close, dev, half, host, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# widths of every thread count; rows that a workgroup's do not divide, odd and even numbers of them a workgroup
NORM = [(4101, 520), (2053, 64), (6200, 1024), (1537, 1100), (1024, 2048), (1537, 4096), (777, 4100), (777, 8192), (1025, 8200), (777, 16383)]


@pytest.mark.parametrize("T,D", NORM)
@pytest.mark.parametrize("dtype,wdtype,with_dh", [("bf16", "f32", True), ("bf16", "bf16", False), ("f32", "f32", True), ("f32", "bf16", False)])
def test_norm_gradient_of_many_rows(T, D, dtype, wdtype, with_dh):
    rng = np.random.default_rng(T + D)
    H, h = dev(rows(rng, T, D), dtype)
    DY, dy = dev(rng.normal(size=(T, D)) * np.exp(rng.normal(size=(T, 1))), dtype)
    DH, dh = dev(rng.normal(size=(T, D)), dtype) if with_dh else (None, None)
    W, w = dev(1 + 0.3 * rng.normal(size=D), wdtype)
    rstd = (1.0 / np.sqrt((h * h).mean(1) + 1e-5)).astype(np.float32)
    rs = rstd.astype(np.float64)
    dx, dw = O.rms_norm_bwd(dy, h, w, rs, dh)
    gdx, gdw = nm.rms_norm_bwd(DY, H, W, torch.from_numpy(rstd).cuda(), dH=DH)
    xh, g = np.abs(h * rs[:, None]), np.abs(dy * w)
    tol = rs[:, None] * (4 * U * g + xh * 70 * U * (g * xh).mean(1, keepdims=True)) + 4 * U * np.abs(dx)
    close(gdx, dx, tol + half(dx, dtype) * 1.01 + (0 if dh is None else 2 * U * np.abs(dh)), "dx")
    per = 512 * 4 if D <= 1024 else 512 if D <= 4096 else 256      # rows that the call's workgroups take at once
    close(gdw, dw, (T / per + 1 + 4 + 32 + 16 + 4) * U * (np.abs(dy) * xh).sum(0) + 1e-37, "dw")
    again = nm.rms_norm_bwd(DY, H, W, torch.from_numpy(rstd).cuda(), dH=DH)
    assert torch.equal(again[0], gdx) and torch.equal(again[1], gdw)
