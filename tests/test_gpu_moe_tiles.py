"""The 8-bit products and quantisers at the sizes that take their large forms (GPU): the 256 x 256 tiles, which
only bf16 results of more than 512 small tiles take, and the quantiser of four rows a wave.

Products of small integers whose scales are powers of two are exact in every sum (below 2^24 of the
smallest unit), so a bf16 result is the exact value rounded once and is compared bit for bit.
Quantisation is exact.
"""

import numpy as np
import pytest
import torch

import sparse_matmul_ffns_amd as nm
from oracle import moe_oracle as MO
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
T8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _large(M, N, E=1):
    """The choice of 256 x 256 tiles for a bf16 result of more than 64 rows a group (fp8_gemm.hip, run())."""
    tiles = lambda b: -(-M // b) * -(-N // b) * E
    return -(-tiles(256) // 256) * 5 <= -(-tiles(128) // 512) * 3


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def matrix(self, fmt, *shape, ld=None):
        """Integers -3 .. 3; `ld` bytes a row, NaN behind the columns."""
        v = torch.randint(-3, 4, shape, generator=self.g, device="cuda").float()
        ld = shape[-1] if ld is None else ld
        wide = torch.full((*shape[:-1], ld), 0x7F, dtype=torch.uint8, device="cuda").view(T8[fmt])
        wide[..., :shape[-1]] = v.to(T8[fmt])
        return wide[..., :shape[-1]], v.double()

    def scales(self, *shape):
        return 2.0 ** torch.randint(-3, 3, shape, generator=self.g, device="cuda").float()


def _by_rows(v, s):
    return v * s.double().t().repeat_interleave(128, 1)[:, :v.shape[1]]


def _by_blocks(v, s):
    return v * s.double().repeat_interleave(128, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]


def _rounded(ref):
    f = ref.float()
    assert bool((f.double() == ref).all())       # exact in fp32
    return f.bfloat16()


@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,K", [(3000, 3300, 1040), (2561, 3457, 1001), (4100, 2060, 100), (2900, 3330, 2048)])
def test_large_tiles(M, N, K, block, fa, fb):
    """Partial tiles at both ends, K ending inside a block, a first and only stage that is also the last."""
    assert _large(M, N)
    d = Draw(M + block)
    ld, Kb = -(-K // 16) * 16, -(-K // 128)
    (A, a), (B, b) = d.matrix(fa, M, K, ld=ld), d.matrix(fb, N, K, ld=ld)
    sa, sb = d.scales(Kb, M), d.scales(Kb, N) if block == 1 else d.scales(-(-N // 128), Kb)
    want = _rounded(_by_rows(a, sa) @ (_by_rows(b, sb) if block == 1 else _by_blocks(b, sb)).t())
    for _ in range(2):
        C = nm.fp8_gemm_nt(A, sa, B, sb, b_block=block)
        assert torch.equal(C, want)


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("K,head,tail", [(1168, 0, 0), (1000, 300, 513), (128, 1, 0)])
def test_large_tiles_of_uneven_groups(K, head, tail, fa):
    """Groups of one row to thousands (waves of a partial tile that only load), empty ones, rows before
    the first group and behind the last."""
    counts = [1, 2500, 0, 37, 256, 255, 257, 3000, 64, 65, 0, 0, 1900, 129, 4000, 3, 1200, 700, 0, 1200]
    E, N = len(counts), 1024
    off = np.concatenate([[head], head + np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1]) + tail
    assert _large(rows, N) and rows // E > 64
    d = Draw(K + head)
    ld, Kb = -(-K // 16) * 16, -(-K // 128)
    (A, a), (B, b) = d.matrix(fa, rows, K, ld=ld), d.matrix("e4m3", E, N, K, ld=ld)
    sa, sb = d.scales(Kb, rows), d.scales(E, N // 128, Kb)
    ref, va = torch.zeros(rows, N, dtype=torch.float64, device="cuda"), _by_rows(a, sa)
    for e in range(E):
        ref[off[e]:off[e + 1]] = va[off[e]:off[e + 1]] @ _by_blocks(b[e], sb[e]).t()
    want = _rounded(ref)
    for _ in range(2):
        assert torch.equal(nm.fp8_gemm_nt_grouped(A, sa, B, sb, torch.from_numpy(off).cuda()), want)


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
def test_large_tiles_of_reduction_groups(fa):
    counts = [128, 0, 1280, 256, 0, 384, 128, 640]
    E, M, N = len(counts), 1300, 1200
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1])
    assert _large(M, N, E)
    d = Draw(7)
    (A, a), (B, b) = d.matrix(fa, M, rows), d.matrix("e4m3", N, rows)
    sa, sb = d.scales(rows // 128, M), d.scales(rows // 128, N)
    va, vb = _by_rows(a, sa), _by_rows(b, sb)
    C = nm.fp8_gemm_nt_grouped_k(A, sa, B, sb, torch.from_numpy(off).cuda(), out_dtype=torch.bfloat16)
    for e in range(E):
        assert torch.equal(C[e], _rounded(va[:, off[e]:off[e + 1]] @ vb[:, off[e]:off[e + 1]].t()))


# ---- the quantiser of four rows a wave -----------------------------------------------------------
def _quantize(x, fmt):
    """MO.quantize, for many rows at once."""
    R, K = x.shape
    Kb = -(-K // 128)
    p = np.zeros((R, Kb * 128))
    p[:, :K] = x
    p = p.reshape(R, Kb, 128)
    amax = np.where(np.isfinite(p), np.abs(p), 0.0).max(2)
    e = np.ceil(np.log2(np.where(amax > 0, amax, 1.0) / MO.MAX8[fmt]))
    s = 2.0 ** np.maximum(e, -126)                     # near it, then the smallest that holds amax
    s = np.where(s * MO.MAX8[fmt] < amax, 2 * s, s)
    s = np.where((s / 2 * MO.MAX8[fmt] >= amax) & (s > 2.0 ** -126), s / 2, s)
    s = np.where(amax > 0, s, 1.0)
    return MO.encode8(p / s[:, :, None], fmt).reshape(R, Kb * 128), np.ascontiguousarray(s.T)


def _wild(rng, R, K, dtype):
    x = rng.normal(size=(R, K)) * np.exp(rng.normal(size=(R, 1)) * 4) * np.exp(rng.normal(size=(1, K)))
    x[rng.random((R, K)) < 0.1] = 0.0
    x[R // 2] = 0.0
    bad = rng.integers(0, R, size=40), rng.integers(0, K, size=40)
    x[bad] = np.resize([np.nan, np.inf, -np.inf], 40)
    x[3] = 1e-42 if dtype == "f32" else 1e-39           # subnormal
    x[-1] = 448.0 * 2.0 ** 5
    x[-1, -1] = 449.0 * 2.0 ** 5 if dtype == "f32" else 452.0 * 2.0 ** 5
    x[-2, -1] = np.nan
    return x


def _device(a, dtype, pad):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    wide = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=t.dtype)
    wide[:, :a.shape[1]] = t
    return wide.cuda()[:, :a.shape[1]], t.double().numpy()


def test_quantize_of_many_rows_matches_the_oracle():
    x = _wild(np.random.default_rng(1), 20, 300, "f32").astype(np.float32).astype(np.float64)
    for fmt in T8:
        for p, q in zip(_quantize(x, fmt), MO.quantize(x, fmt)):
            assert np.array_equal(p, q)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype,pad,gather,gated", [("bf16", 0, False, False), ("f32", 0, True, False), ("bf16", 8, True, True),
                                                    ("bf16", 3, False, True), ("f32", 1, True, True), ("f32", 0, False, True)])
@pytest.mark.parametrize("R,K", [(8203, 264), (2101, 2056)])
def test_quantize_many_rows(R, K, dtype, pad, gather, gated, fmt):
    rng = np.random.default_rng(R + K + pad)
    assert -(-R // 16) * -(-K // 512) >= 512 and R % 16 != 0        # four rows a wave, a remainder
    div = 3
    dx, x = _device(_wild(rng, R // div + 7 if gather else R, K, dtype), dtype, pad)
    src = rng.integers(-1, x.shape[0] * div + 4, size=R).astype(np.int32) if gather else None
    g, dg = None, None
    if gated:
        dg, g = (dx, x) if not gather else _device(rng.normal(size=(R, K)), dtype, pad)
    y = MO.rows_of(x, src, div, g)
    kw = dict(src=None if src is None else torch.from_numpy(src).cuda(), div=div if gather else 1, gate=dg)
    for t in (False, True):
        want, ws = _quantize(np.ascontiguousarray(y.T) if t else y, fmt)
        q, s = (nm.fp8_quantize_t if t else nm.fp8_quantize)(dx, T8[fmt], **kw)
        assert np.array_equal(s.double().cpu().numpy(), ws)
        v = MO.decode8(fmt)
        a, b = v[q.cpu().view(torch.uint8).numpy()], v[want]
        assert np.array_equal(a, b, equal_nan=True)
        assert np.array_equal(np.signbit(a)[~np.isnan(a)], np.signbit(b)[~np.isnan(b)])
