"""Pins of the mixture-of-experts oracle (CPU): the 8-bit formats against torch's, the routing gradient
against differences, and the calls' refusals, which the host makes before anything is launched."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import moe_oracle as MO
from sparse_matmul_ffns_amd import nmsparse as nm

FAKE = 4096   # a non-NULL address that is never dereferenced
T8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_decode_matches_torch(fmt):
    b = torch.arange(256, dtype=torch.uint8)
    want = b.view(T8[fmt]).double().numpy()
    got = MO.decode8(fmt)
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_encode_rounds_to_nearest_even(fmt):
    vals = MO.decode8(fmt)[:128]
    vals = vals[np.isfinite(vals)]
    mid = (vals[:-1] + vals[1:]) / 2
    codes = MO.encode8(mid, fmt)
    assert (codes % 2 == 0).all()                                    # ties to the even byte
    eps = np.spacing(mid)
    assert np.array_equal(MO.encode8(mid - eps, fmt), np.arange(mid.size))
    assert np.array_equal(MO.encode8(mid + eps, fmt), np.arange(1, mid.size + 1))
    assert np.array_equal(MO.encode8(-vals, fmt), np.arange(vals.size) | 0x80)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_block_scale_is_the_smallest_power(fmt):
    for amax in (1.0, MAX := MO.MAX8[fmt], np.nextafter(MAX, np.inf), 2 * MAX, 1e-30, 3e38, 1e-45):
        s = MO.block_scale(np.array([amax, -amax / 3, 0.0]), fmt)
        assert amax / s <= MAX and (s == 2.0 ** -126 or amax / (s / 2) > MAX)
    assert MO.block_scale(np.zeros(128), fmt) == 1.0
    assert MO.block_scale(np.array([np.inf, np.nan, 1.0]), fmt) == MO.block_scale(np.array([1.0]), fmt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_matches_differences(score, renorm):
    rng = np.random.default_rng(5)
    l = rng.normal(size=(3, 11))
    ids, w, _ = MO.route(l, 4, score, renorm=renorm, scale=1.7)
    dw = rng.normal(size=ids.shape)
    dl = MO.route_bwd(l, ids, w, dw, score, renorm, 1.7)
    h = 1e-5
    for e in range(l.shape[1]):
        up, dn = l.copy(), l.copy()
        up[:, e] += h
        dn[:, e] -= h
        diff = ((MO.route_weights_of(up, ids, score, renorm, 1.7) - MO.route_weights_of(dn, ids, score, renorm, 1.7))
                * dw).sum(1) / (2 * h)
        assert np.allclose(dl[:, e], diff, rtol=1e-7, atol=1e-9)


def test_combine_gradient_matches_differences():
    rng = np.random.default_rng(6)
    O, dY = rng.normal(size=(7, 5)), rng.normal(size=(3, 5))
    pos = np.array([[0, 3], [6, -1], [2, 5]])
    w = rng.normal(size=pos.shape)
    dO, dw = MO.combine_bwd(dY, O, pos, w)
    loss = lambda O_, w_: (MO.combine(O_, pos, w_) * dY).sum()
    h = 1e-6
    for i in np.ndindex(O.shape):
        up, dn = O.copy(), O.copy()
        up[i] += h
        dn[i] -= h
        assert abs((loss(up, w) - loss(dn, w)) / (2 * h) - dO[i]) < 1e-8
    for i in np.ndindex(w.shape):
        up, dn = w.copy(), w.copy()
        up[i] += h
        dn[i] -= h
        assert abs((loss(O, up) - loss(O, dn)) / (2 * h) - dw[i]) < 1e-8


# ---- refusals ---------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def L():
    return nm.lib()


def test_route_errors(L):
    # dt, logits, ldl, T, E, score, bias, groups, topk_groups, group_top, k, renorm, scale, ids, weights, stream
    def call(dt=1, logits=FAKE, ldl=64, T=4, E=64, score=0, bias=None, groups=1, tg=1, gt=2, k=8, scale=1.0, ids=FAKE,
             w=FAKE):
        return L.moe_route(dt, logits, ldl, T, E, score, bias, groups, tg, gt, k, 1, scale, ids, w, None)
    assert call(logits=None) == call(ids=None) == call(w=None) == nm.NM_ERR_NULL
    for bad in (dict(dt=3), dict(score=2), dict(E=1025, ldl=1025), dict(k=65), dict(groups=65), dict(gt=0), dict(gt=3),
                dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(**bad) == nm.NM_ERR_UNSUPPORTED, bad
    for bad in (dict(T=0), dict(E=0), dict(k=0), dict(ldl=63), dict(groups=7), dict(groups=4, tg=5), dict(groups=4, tg=0),
                dict(groups=16, tg=1, k=5), dict(E=4, k=8), dict(T=1 << 29)):
        assert call(**bad) == nm.NM_ERR_SHAPE, bad
    for bad in (dict(logits=FAKE + 1), dict(bias=FAKE + 2), dict(ids=FAKE + 1), dict(w=FAKE + 2)):
        assert call(**bad) == nm.NM_ERR_ALIGN, bad
    # dt, logits, ldl, T, E, score, k, renorm, scale, ids, weights, dweights, dlogits, lddl, stream
    assert L.moe_route_bwd(1, FAKE, 64, 4, 64, 0, 8, 1, 1.0, FAKE, FAKE, None, FAKE, 64, None) == nm.NM_ERR_NULL
    assert L.moe_route_bwd(1, FAKE, 64, 4, 64, 0, 65, 1, 1.0, FAKE, FAKE, FAKE, FAKE, 64, None) == nm.NM_ERR_UNSUPPORTED
    assert L.moe_route_bwd(1, FAKE, 64, 4, 64, 0, 8, 1, 1.0, FAKE, FAKE, FAKE, FAKE, 63, None) == nm.NM_ERR_SHAPE
    assert L.moe_route_bwd(1, FAKE, 64, 4, 4, 0, 8, 1, 1.0, FAKE, FAKE, FAKE, FAKE, 64, None) == nm.NM_ERR_SHAPE
    assert L.moe_route_bwd(0, FAKE, 64, 4, 64, 0, 8, 1, 1.0, FAKE, FAKE, FAKE, FAKE + 2, 64, None) == nm.NM_ERR_ALIGN


def test_plan_errors(L):
    need = ctypes.c_int64(7)
    assert L.moe_plan_work_bytes(16, 8, 64, ctypes.byref(need)) == nm.NM_OK and need.value == 0
    assert L.moe_plan_work_bytes(8192, 8, 64, ctypes.byref(need)) == nm.NM_OK and need.value > 0
    assert L.moe_plan_work_bytes(8192, 8, 64, None) == nm.NM_ERR_NULL
    assert L.moe_plan_work_bytes(0, 8, 64, ctypes.byref(need)) == nm.NM_ERR_SHAPE
    # ids, T, k, E, align, offsets, counts, src, rows, pos, work, work_bytes, stream
    def call(ids=FAKE, T=16, k=8, E=64, align=1, off=FAKE, cnt=FAKE, src=FAKE, rows=128, pos=FAKE, work=None, wb=0):
        return L.moe_plan(ids, T, k, E, align, off, cnt, src, rows, pos, work, wb, None)
    assert call(ids=None) == call(off=None) == call(cnt=None) == call(src=None) == call(pos=None) == nm.NM_ERR_NULL
    assert call(T=8192, rows=65536) == nm.NM_ERR_NULL                   # work memory needed
    assert call(T=8192, rows=65536, work=FAKE, wb=16) == nm.NM_ERR_SHAPE
    assert call(rows=127) == nm.NM_ERR_SHAPE
    assert call(align=16, rows=128 + 64 * 15 - 1) == nm.NM_ERR_SHAPE
    assert call(align=3) == call(align=512) == call(E=1025) == call(k=65) == nm.NM_ERR_UNSUPPORTED
    assert call(T=0) == call(E=0) == call(rows=1 << 31) == nm.NM_ERR_SHAPE
    assert call(src=FAKE + 2) == nm.NM_ERR_ALIGN


def test_quantize_errors(L):
    # dt, X, ldx, RX, src, div, gate, ldg, R, K, fmt, Q, ldq, S, lds, stream
    def call(f=L.fp8_quantize, dt=1, X=FAKE, ldx=200, RX=8, src=None, div=1, gate=None, ldg=0, R=8, K=200, fmt=0, Q=FAKE,
             ldq=256, S=FAKE, lds=256):
        return f(dt, X, ldx, RX, src, div, gate, ldg, R, K, fmt, Q, ldq, S, lds, None)
    assert call(X=None) == call(Q=None) == call(S=None) == nm.NM_ERR_NULL
    assert call(dt=2) == call(fmt=2) == nm.NM_ERR_UNSUPPORTED
    for bad in (dict(R=0), dict(K=0), dict(RX=0), dict(ldx=199), dict(R=9), dict(src=FAKE, div=0), dict(gate=FAKE, ldg=199),
                dict(ldq=255), dict(lds=7)):
        assert call(**bad) == nm.NM_ERR_SHAPE, bad
    assert call(X=FAKE + 1) == call(src=FAKE + 2) == call(gate=FAKE + 1, ldg=200) == call(S=FAKE + 2) == nm.NM_ERR_ALIGN
    assert call(f=L.fp8_quantize_t, ldq=127) == nm.NM_ERR_SHAPE
    assert call(f=L.fp8_quantize_t, lds=199) == nm.NM_ERR_SHAPE
    # dt, W, ldw, E, N, K, fmt, Q, ldq, S, Qt, ldqt, St, stream
    assert L.fp8_quantize_weight(1, FAKE, 64, 2, 32, 64, 0, FAKE, 128, FAKE, FAKE, 128, None, None) == nm.NM_ERR_NULL
    assert L.fp8_quantize_weight(1, FAKE, 64, 2, 32, 64, 0, FAKE, 127, FAKE, None, 0, None, None) == nm.NM_ERR_SHAPE
    assert L.fp8_quantize_weight(1, FAKE, 64, 2, 32, 64, 0, FAKE, 128, FAKE, FAKE, 127, FAKE, None) == nm.NM_ERR_SHAPE
    assert L.fp8_quantize_weight(1, FAKE, 64, 0, 32, 64, 0, FAKE, 128, FAKE, None, 0, None, None) == nm.NM_ERR_SHAPE


def test_gemm_errors(L):
    # fa, A, lda, sa, ldsa, fb, B, ldb, sb, ldsb, b_block, M, N, K, out, C, ldc, stream
    def call(fa=0, A=FAKE, lda=256, sa=FAKE, ldsa=8, fb=0, B=FAKE, ldb=256, sb=FAKE, ldsb=2, bb=128, M=8, N=16, K=256,
             out=1, C=FAKE, ldc=16):
        return L.fp8_gemm_nt(fa, A, lda, sa, ldsa, fb, B, ldb, sb, ldsb, bb, M, N, K, out, C, ldc, None)
    assert call(A=None) == call(sa=None) == call(B=None) == call(sb=None) == call(C=None) == nm.NM_ERR_NULL
    assert call(fa=2) == call(fb=-1) == call(out=2) == call(bb=64) == nm.NM_ERR_UNSUPPORTED
    for bad in (dict(M=0), dict(N=0), dict(K=0), dict(lda=255), dict(ldb=255), dict(ldsa=7), dict(ldsb=1), dict(ldc=15),
                dict(bb=1, ldsb=15)):
        assert call(**bad) == nm.NM_ERR_SHAPE, bad
    assert call(sa=FAKE + 2) == call(sb=FAKE + 1) == call(C=FAKE + 1) == nm.NM_ERR_ALIGN
    # ..., sb, ldsb, offsets, E, rows, N, K, out, C, ldc, stream
    g = L.fp8_gemm_nt_grouped
    assert g(0, FAKE, 256, FAKE, 8, 0, FAKE, 256, FAKE, 2, None, 4, 8, 16, 256, 1, FAKE, 16, None) == nm.NM_ERR_NULL
    assert g(0, FAKE, 256, FAKE, 8, 0, FAKE, 256, FAKE, 2, FAKE, 1025, 8, 16, 256, 1, FAKE, 16, None) == \
        nm.NM_ERR_UNSUPPORTED
    assert g(0, FAKE, 256, FAKE, 8, 0, FAKE, 256, FAKE, 1, FAKE, 4, 8, 16, 256, 1, FAKE, 16, None) == nm.NM_ERR_SHAPE
    # ..., sb, ldsb, offsets, E, M, N, rows, out, C, ldc, stream
    k = L.fp8_gemm_nt_grouped_k
    assert k(0, FAKE, 256, FAKE, 8, 0, FAKE, 256, FAKE, 16, None, 4, 8, 16, 256, 1, FAKE, 16, None) == nm.NM_ERR_NULL
    assert k(0, FAKE, 256, FAKE, 8, 0, FAKE, 256, FAKE, 16, FAKE, 4, 8, 16, 200, 1, FAKE, 16, None) == nm.NM_ERR_SHAPE
    assert k(0, FAKE, 256, FAKE, 8, 0, FAKE, 256, FAKE, 15, FAKE, 4, 8, 16, 256, 1, FAKE, 16, None) == nm.NM_ERR_SHAPE
    assert k(0, FAKE, 256, FAKE, 8, 0, FAKE, 256, FAKE, 16, FAKE + 2, 4, 8, 16, 256, 1, FAKE, 16, None) == nm.NM_ERR_ALIGN


def test_combine_errors(L):
    # dt, O, ldo, rows, pos, weights, T, k, D, Y, ldy, stream
    def call(dt=1, O=FAKE, ldo=64, rows=8, pos=FAKE, w=None, T=2, k=4, D=64, Y=FAKE, ldy=64):
        return L.moe_combine(dt, O, ldo, rows, pos, w, T, k, D, Y, ldy, None)
    assert call(O=None) == call(pos=None) == call(Y=None) == nm.NM_ERR_NULL
    assert call(dt=2) == call(k=65) == nm.NM_ERR_UNSUPPORTED
    assert call(T=0) == call(k=0) == call(D=0) == call(rows=0) == call(ldo=63) == call(ldy=63) == nm.NM_ERR_SHAPE
    assert call(O=FAKE + 1) == call(pos=FAKE + 2) == call(w=FAKE + 2) == nm.NM_ERR_ALIGN
    # dt, dY, lddy, O, ldo, rows, src, pos, weights, T, k, D, dO, lddo, dweights, stream
    b = L.moe_combine_bwd
    assert b(1, FAKE, 64, FAKE, 64, 8, FAKE, FAKE, None, 2, 4, 64, FAKE, 64, FAKE, None) == nm.NM_ERR_NULL
    assert b(1, FAKE, 64, FAKE, 64, 8, FAKE, FAKE, FAKE, 2, 4, 64, FAKE, 63, FAKE, None) == nm.NM_ERR_SHAPE
    assert b(1, FAKE, 64, FAKE, 64, 8, FAKE, FAKE, FAKE, 2, 4, 64, FAKE, 64, FAKE + 2, None) == nm.NM_ERR_ALIGN


def test_binding_refuses():
    x = torch.zeros(4, 64)
    for call in (lambda: nm.moe_route(x, 2), lambda: nm.moe_plan(torch.zeros(2, 2, dtype=torch.int32), 4),
                 lambda: nm.fp8_quantize(x), lambda: nm.fp8_quantize_t(x), lambda: nm.fp8_quantize_weight(x),
                 lambda: nm.moe_combine(x, torch.zeros(2, 2, dtype=torch.int32))):
        with pytest.raises(ValueError):      # CPU tensors
            call()
    assert nm.moe_plan_rows(128, 64, 1) == 128 and nm.moe_plan_rows(8, 64, 128) == 1024
