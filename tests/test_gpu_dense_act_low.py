"""The activations where the sigmoid leaves fp32's normal numbers (GPU).

Above -87.3 the sigmoid is normal and its relative error is below (|x| + 3) 2^-23, the product's half a step more.  Below, the kernels' sigmoid is
0 and the exact one less than 2^-126, so x sigmoid(x) is off by less than 88 2^-126 = 1.04e-36 (|x| e^x falls from there on), and
the derivative s + x s (1 - s) by less than 89 2^-126; GELU reaches that region at x = -10.0 (2 u = -87.3)."""

import numpy as np
import pytest
import torch

import sparse_matmul_ffns_amd as nm
from oracle import dense_oracle as O
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("kind,lo,hi", [("silu", -110.0, -80.0), ("gelu_tanh", -12.0, -8.0)])
def test_beside_and_below_the_border(kind, lo, hi):
    require_gpu()
    z = torch.linspace(lo, hi, 4096, dtype=torch.float64).bfloat16().view(16, 256)
    z64 = z.double().numpy()
    eye = torch.eye(16).bfloat16().cuda()
    got = nm.linear_fwd(eye, z.t().contiguous().cuda(), act=kind, out_dtype=torch.float32).double().cpu().numpy()
    x = O._arg(z64, kind)
    s = O.sigmoid(x)
    normal = x > -87.3
    assert normal.any() and (~normal).any()
    want = O.act(z64, kind)
    err = np.abs(got - want)
    # the argument x carries four roundings in front of the exponential (GELU's polynomial)
    assert (err[normal] <= ((2 * np.abs(x) + 6 + (8 * np.abs(x) if kind == "gelu_tanh" else 0)) * U * np.abs(want) + 2.0 ** -149)[normal]).all()
    assert (err[~normal] <= 88 * 2.0 ** -126).all() and (got[~normal] <= 0).all()
    d = nm.linear_bwd_act(torch.ones_like(z).cuda(), z.cuda(), act=kind, dZ=torch.empty_like(z).cuda())[0].double().cpu().numpy()
    q = 2 * O.GK * (1 + 3 * O.CUBE * z64 * z64) if kind == "gelu_tanh" else np.ones_like(z64)
    bound = (2.0 ** -8 + 2 ** -15) * np.abs(O.dact(z64, kind)) + np.where(normal, 0, (1 + np.abs(z64) * q) * 2.0 ** -126) + 2.0 ** -133
    assert (np.abs(d - O.dact(z64, kind)) <= bound).all()
    assert (s[~normal] < 2.0 ** -125.8).all()
