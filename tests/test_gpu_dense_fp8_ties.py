"""rms_norm_fp8's one rounding (GPU): bytes and scales against 64 bits, equal everywhere.

y = (x + r) rstd w is irrational, so it lies beside a border between two 8-bit values, not on it; fp32's nearest value to y
may lie on it, and rounding that takes the even neighbour whichever side y is on.  The inputs hold such elements (the test asserts it), and
sums x + r that fp32 does not hold.

Both sides compute in 64 bits.  A sum of D squares is off by D 2^-53 of itself at most, the root by half of that, the products by a few
2^-53: for D up to 16384 the two may differ by 2^-39 + 2^-39 of y.  Elements that lie within 2^-38 of themselves beside a border are left out
(expected: 1e-4 of an element in these tests).
"""

import numpy as np
import pytest
import torch

import sparse_matmul_ffns_amd as nm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
T8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def blocks(y, fmt):
    """y [T, D] float64 -> (values / scale [T, Dp / 128, 128], scale [T, Dp / 128])."""
    T, D = y.shape
    full = np.zeros((T, -(-D // 128) * 128))
    full[:, :D] = y
    full = full.reshape(T, -1, 128)
    peak = np.abs(full).max(2)
    m, e = np.frexp(peak / TOP[fmt])          # the smallest power of two that is at least the quotient
    scale = np.where(peak > 0, np.ldexp(1.0, np.maximum(np.where(m > 0.5, e, e - 1), -126)), 1.0)
    return full / scale[:, :, None], scale


def round8(v, fmt):
    """v to the nearest 8-bit value, ties to even; and v's distance from the nearest border, relative to v."""
    digits, lowest = (3, -6) if fmt == "e4m3" else (2, -14)
    step = np.ldexp(1.0, np.maximum(np.frexp(v)[1] - 1, lowest) - digits)
    q = v / step
    return np.rint(q) * step, np.abs(np.abs(q - np.floor(q)) - 0.5) / np.maximum(np.abs(q), 1e-300)


CASES = [("bf16", "f32", 2048, 2048, 0), ("bf16", "bf16", 2048, 2048, 16), ("f32", "f32", 2600, 2050, 0), ("f32", "f32", 257, 16384, 12),
         ("bf16", "f32", 3000, 520, None), ("f32", "bf16", 1900, 4099, None)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype,wdtype,T,D,shift", CASES)
def test_bytes_are_the_64_bit_ones(dtype, wdtype, T, D, shift, fmt):
    """shift: the residual is 2^-shift of x (None: no residual)."""
    g = torch.Generator().manual_seed(T + D)
    wide = lambda: torch.randn(T, D, generator=g) * torch.exp(0.5 * torch.randn(T, 1, generator=g)) * torch.exp(0.5 * torch.randn(1, D, generator=g))
    X = wide().to(TD[dtype])
    R = None if shift is None else (wide() * 2.0 ** -shift).to(TD[dtype])
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(TD[wdtype])
    h = X.double().numpy() + (0.0 if R is None else R.double().numpy())
    eps = float(np.float32(1e-5))
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w.double().numpy()
    v, scale = blocks(y, fmt)
    want, margin = round8(v, fmt)
    # elements that the nearest fp32 value sends to another byte
    twice = round8(blocks(y.astype(np.float32).astype(np.float64), fmt)[0], fmt)[0]
    assert (twice != want).sum() >= 1
    if shift is not None:
        assert (h != h.astype(np.float32)).any()
    Q, S, _, _ = nm.rms_norm_fp8(X.cuda(), w.cuda(), eps=eps, residual=None if R is None else R.cuda(), fmt=T8[fmt])
    peak = np.abs(v).max(2) / TOP[fmt]        # in (0.5, 1]: beside 1 or 0.5 the next scale begins
    clear = (np.abs(peak - 1) > 2.0 ** -38) & (np.abs(peak - 0.5) > 2.0 ** -38)
    got_s = S.cpu().double().numpy().T
    assert np.array_equal(got_s[clear], scale[clear])
    got = Q.float().cpu().double().numpy().reshape(v.shape)
    bad = (got != want) & (margin > 2.0 ** -38) & clear[:, :, None]
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


def test_scales_beside_a_border():
    """The largest magnitude of a block lies beside 448 or 57344 times a power of two by less than fp32 resolves: the scale follows the
    exact value.  A row of +-1 and one larger element a: y of that element is a w rstd; w brings it to the border, and
    its next fp32 neighbours to both sides of it."""
    D = 128
    x = torch.ones(64, D)
    x[:, 7] = 1 + torch.arange(64) / 64.0
    eps = float(np.float32(1e-5))
    h = x.double().numpy()
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    for fmt in ("e4m3", "e5m2"):
        for t in range(64):
            near = np.float32(0.875 / (h[t, 7] * rstd[t]))
            for w7 in (np.nextafter(near, np.float32(0)), near, np.nextafter(near, np.float32(9))):
                w = torch.full((D,), 0.25)
                w[7] = float(w7)
                y = h[t:t + 1] * rstd[t] * w.double().numpy()
                assert abs(y[0, 7] / 0.875 - 1) < 2.0 ** -22
                _, scale = blocks(y, fmt)
                if t % 8 == 0 or abs(y[0, 7] / 0.875 - 1) < 2.0 ** -25:
                    _, S, _, _ = nm.rms_norm_fp8(x[t:t + 1].cuda(), w.cuda(), eps=eps, fmt=T8[fmt])
                    assert float(S[0, 0]) == scale[0, 0], (fmt, t, float(w7))


def test_values_that_are_exact_and_not_finite():
    """Rows whose y is an 8-bit value or exactly between two (ties go to even), zeros of both signs, infinities and NaN."""
    D = 256
    x = torch.zeros(4, D)
    x[0] = 2.0                                   # mean of squares 4, and eps 12: rstd 1/4, y = w / 2
    x[1, :128] = -2.0
    x[1, 128:] = 2.0
    x[2] = 2.0
    x[2, 3] = float("inf")
    x[3] = 2.0
    x[3, 5] = float("nan")
    w = torch.full((D,), 2.0)
    w[:16] = 2 + torch.arange(16) / 8.0          # y = 1 .. 1.9375 by sixteenths: e4m3 holds every second one
    Q, S, _, rstd = nm.rms_norm_fp8(x.cuda(), w.cuda(), eps=12.0)
    got = (Q.float().cpu() * S.cpu().t().repeat_interleave(128, 1)).double().numpy()
    assert rstd[0] == 0.25
    y = x.double().numpy()[:2] * 0.25 * w.double().numpy()
    v, scale = blocks(y, "e4m3")
    assert np.array_equal(got[:2], (round8(v, "e4m3")[0] * scale[:, :, None]).reshape(2, D))
    assert np.isnan(got[2, 3]) and (np.delete(got[2], 3) == 0).all() and np.isnan(got[3]).all()


@pytest.mark.parametrize("dtype,wdtype,T,D,shift", CASES)
def test_the_result_beside_the_bytes_is_rounded_once(dtype, wdtype, T, D, shift):
    """Y in bf16 or fp32 against 64 bits rounded once; the margin as above."""
    g = torch.Generator().manual_seed(T + D + 1)
    X = torch.randn(T, D, generator=g).to(TD[dtype])
    R = None if shift is None else (torch.randn(T, D, generator=g) * 2.0 ** -shift).to(TD[dtype])
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(TD[wdtype])
    h = X.double().numpy() + (0.0 if R is None else R.double().numpy())
    eps = float(np.float32(1e-5))
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w.double().numpy()
    digits = 7 if dtype == "bf16" else 23
    step = np.ldexp(1.0, np.frexp(y)[1] - 1 - digits)
    q = y / step
    want, margin = np.rint(q) * step, np.abs(np.abs(q - np.floor(q)) - 0.5) / np.maximum(np.abs(q), 1e-300)
    if dtype == "bf16":
        assert (torch.from_numpy(y).float().bfloat16().double().numpy() != want).any()     # by way of fp32 some differ
    Y = torch.empty(T, D, dtype=TD[dtype], device="cuda")
    nm.rms_norm_fp8(X.cuda(), w.cuda(), eps=eps, residual=None if R is None else R.cuda(), Y=Y)
    bad = (Y.double().cpu().numpy() != want) & (margin > 2.0 ** -38)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [96, 2048, 9000])
def test_rows_of_any_size(dtype, D):
    """Rows from 2^-100 to 2^127, whose squares fp32 does not hold, and sums that it does not hold."""
    g = torch.Generator().manual_seed(D)
    T = 40
    size = torch.linspace(-100, 125, T).round()
    X = (torch.randn(T, D, generator=g).clamp(-3.5, 3.5) * torch.exp2(size)[:, None]).to(TD[dtype])
    w = 1 + 0.2 * torch.randn(D, generator=g)
    for R in (None, X.clone()):                  # the last rows' doubles are beyond fp32
        h = X.double().numpy() * (1 if R is None else 2)
        for eps in (1e-5, 1e-38):
            eps = float(np.float32(eps))
            rstd = 1 / np.sqrt((h * h).mean(1) + eps)
            y = h * rstd[:, None] * w.double().numpy()
            Q, S, _, got = nm.rms_norm_fp8(X.cuda(), w.cuda(), eps=eps, residual=None if R is None else R.cuda())
            # half a step of fp32: relative, and below 2^-126 (rows beyond 2^126) half of the subnormals' step of 2^-149
            assert (np.abs(got.double().cpu().numpy() - rstd) <= np.maximum(2.0 ** -24 * rstd, 2.0 ** -150)).all()
            v, scale = blocks(y, "e4m3")
            want, margin = round8(v, "e4m3")
            assert np.array_equal(S.cpu().double().numpy().T, scale)
            # below fp32's normal numbers y is rounded twice
            plain = (np.abs(y) >= 2.0 ** -126)
            plain = np.pad(plain, ((0, 0), (0, -D % 128)), constant_values=True).reshape(v.shape)
            bad = (Q.float().cpu().double().numpy().reshape(v.shape) != want) & (margin > 2.0 ** -38) & plain
            assert not bad.any(), (eps, np.argwhere(bad)[:4].tolist())
