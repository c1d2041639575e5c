"""Outputs of the dense block's calls that meet an input, another output or work memory are refused, those that the header allows and
those that only interleave are not (C ABI; CPU: what passes the checks ends at its first launch, since no GPU is visible)."""

import ctypes
import os
import random

import pytest

from sparse_matmul_ffns_amd import nmsparse as nm

pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="runs only where no GPU is visible: the addresses are made up")
SHAPE, PASSED = nm.NM_ERR_SHAPE, nm.NM_ERR_HIP


@pytest.fixture(scope="module")
def L():
    return nm.lib()


def _bytes(at, rows, cols, ld, es):
    return {at + (r * ld + c) * es + b for r in range(rows) for c in range(cols) for b in range(es)}


def test_any_two_matrices(L):
    """Random places of two small matrices against the sets of their bytes."""
    rng = random.Random(0)
    met = 0
    for _ in range(6000):
        M, N = rng.randint(1, 6), rng.randint(1, 5)
        lda = N + rng.choice([0, 0, 1, 3, rng.randint(0, 20)])
        ldb = rng.choice([lda, N + rng.choice([0, 1, 4, rng.randint(0, 40)])])
        a, b = 4096, 4096 + 2 * rng.randint(-60, 60)
        want = bool(_bytes(a, M, N, lda, 2) & _bytes(b, M, N, ldb, 2)) and not (a == b and (lda == ldb or M == 1))
        got = L.linear_bwd_act(1, a, lda, None, 0, 0, M, N, b, ldb, None, None, 0, None)
        assert got == (SHAPE if want else PASSED), (M, N, lda, ldb, b - a)
        met += want
    assert 1000 < met < 5000
    # matrices of other shapes and types: X [M, K] and dW [N, K] fp32
    for _ in range(6000):
        M, N, K = rng.randint(1, 5), rng.randint(1, 5), rng.randint(1, 5)
        ldx, ldw = K + rng.choice([0, rng.randint(0, 30)]), K + rng.choice([0, rng.randint(0, 30)])
        x, w = 4096 + 2 * rng.randint(0, 1), 4096 + 4 * rng.randint(-60, 40)
        want = bool(_bytes(x, M, K, ldx, 2) & _bytes(w, N, K, ldw, 4))
        got = L.linear_bwd_w(1, 1 << 20, N, x, ldx, M, N, K, 0, 0, w, ldw, None, 0, None)
        assert got == (SHAPE if want else PASSED), (M, N, K, ldx, ldw, x, w)


def test_far_strides(L):
    """Two columns of one buffer with many rows, and rows far apart: neither loops over its rows nor overflows."""
    M, ld = (1 << 31) - 1, 1 << 21
    for off, want in ((16, PASSED), (15, SHAPE), (ld - 16, PASSED), (ld - 15, SHAPE), (5 * ld, SHAPE), (5 * ld + 16, PASSED)):
        assert L.linear_bwd_act(1, 4096, ld, None, 0, 0, M, 16, 4096 + 2 * off, ld, None, None, 0, None) == want, off
    assert L.linear_bwd_act(1, 4096, 1 << 60, None, 0, 0, 5, 16, 4096 + 64, 1 << 60, None, None, 0, None) == PASSED


def _expect(call, base, *cases):
    """Each of `cases`: the addresses (by position) to change, and the status."""
    assert call(*base) == PASSED
    for change, status in cases:
        args = list(base)
        for i, v in change.items():
            args[i] = v
        assert call(*args) == status, change


P = [(1 << 24) * i for i in range(1, 12)]      # places far apart


def test_norm(L):
    # dt, X, ldx, residual, ldr, wdt, w, eps, T, D, H, ldh, Y, ldy, rstd, stream
    X, R, H, Y, w, rstd, Q, S = P[:8]
    base = [1, X, 16, R, 16, 0, w, 1e-5, 4, 16, H, 16, Y, 16, rstd, None]
    _expect(L.rms_norm, base, ({10: X}, PASSED), ({10: R}, PASSED), ({12: X}, PASSED), ({12: R}, PASSED), ({10: R, 12: X}, PASSED),
            ({10: X, 12: R}, PASSED), ({10: X, 12: X}, SHAPE), ({10: R, 12: R}, SHAPE), ({12: H}, SHAPE), ({12: X + 2}, SHAPE),
            ({10: X, 11: 24}, SHAPE), ({10: X + 32}, SHAPE), ({10: X + 128}, PASSED), ({14: Y}, SHAPE), ({14: X + 124}, SHAPE), ({14: X + 128}, PASSED))
    # dt, X, ldx, residual, ldr, wdt, w, eps, T, D, fmt, Q, ldq, S, lds, H, ldh, Y, ldy, rstd, stream
    base = [1, X, 16, R, 16, 0, w, 1e-5, 4, 16, 0, Q, 128, S, 4, H, 16, Y, 16, rstd, None]
    _expect(L.rms_norm_fp8, base, ({15: X}, PASSED), ({17: X}, PASSED), ({15: R, 17: X}, PASSED), ({15: X, 17: X}, SHAPE), ({11: X}, SHAPE),
            ({11: H}, SHAPE), ({13: Q + 508}, SHAPE), ({13: Q + 512}, PASSED), ({13: X}, SHAPE), ({19: S + 12}, SHAPE), ({19: S + 16}, PASSED))
    # dt, dY, lddy, H, ldh, wdt, w, rstd, dH, lddh, T, D, dX, lddx, dw, work, work_bytes, stream
    dY, H, dH, dX, w, rstd, dw, work = P[:8]
    base = [1, dY, 2000, H, 2000, 0, w, rstd, dH, 2000, 4, 2000, dX, 2000, dw, work, 1 << 20, None]
    _expect(L.rms_norm_bwd, base, ({12: dY}, PASSED), ({12: dH}, PASSED), ({12: H}, PASSED), ({12: dY, 13: 2008}, SHAPE), ({12: dH + 4000}, SHAPE),
            ({14: dX}, SHAPE), ({14: dX + 16000}, PASSED), ({15: H}, SHAPE), ({15: dw}, SHAPE))


def test_linear(L):
    # dt, X, ldx, W, ldw, bdt, bias, act, residual, ldr, M, N, K, out, Y, ldy, pre, ldp, work, work_bytes, stream
    X, W, R, Y, pre, bias, work = P[:7]
    base = [1, X, 16, W, 16, 1, bias, 1, R, 16, 4, 16, 16, 1, Y, 16, pre, 16, work, 1 << 16, None]
    _expect(L.linear_fwd, base, ({14: R}, PASSED), ({14: R, 13: 0}, SHAPE), ({14: X}, SHAPE), ({14: W}, SHAPE), ({16: R}, SHAPE), ({16: Y}, SHAPE),
            ({16: X}, SHAPE), ({14: R + 2}, SHAPE), ({14: R, 15: 20}, SHAPE), ({18: Y}, SHAPE), ({18: Y - (1 << 16)}, PASSED), ({18: W}, SHAPE))
    # dt, dY, lddy, pre, ldp, act, M, N, dZ, lddz, db, work, work_bytes, stream
    base = [1, X, 16, W, 16, 2, 4000, 16, Y, 16, R, work, 1 << 20, None]
    _expect(L.linear_bwd_act, base, ({8: X}, PASSED), ({8: W}, PASSED), ({8: X + 32}, SHAPE), ({10: X}, SHAPE), ({10: Y}, SHAPE), ({11: Y}, SHAPE))
    # without an activation pre is not read
    assert L.linear_bwd_act(1, X, 16, W, 16, 0, 4, 16, W + 32, 16, None, None, 0, None) == PASSED
    # dt, dZ, lddz, W, ldw, pre, ldp, act, M, N, K, out, dX, lddx, work, work_bytes, stream
    base = [1, X, 16, W, 16, pre, 16, 1, 4, 16, 16, 1, Y, 16, work, 1 << 16, None]
    _expect(L.linear_bwd_x, base, ({12: pre}, PASSED), ({12: pre, 11: 0}, SHAPE), ({12: X}, SHAPE), ({12: W}, SHAPE), ({14: pre}, SHAPE),
            ({12: pre + 64}, SHAPE))
    # dt, dZ, lddz, X, ldx, M, N, K, accumulate, out, dW, lddw, work, work_bytes, stream
    base = [1, X, 16, R, 16, 4, 16, 16, 0, 1, W, 16, work, 1 << 16, None]
    _expect(L.linear_bwd_w, base, ({10: X}, SHAPE), ({10: R}, SHAPE), ({12: W}, SHAPE), ({10: R + 128}, PASSED))


def test_grad_norm(L):
    dt, ptr, cnt = (ctypes.c_int * 3)(0, 1, 0), (ctypes.c_void_p * 3)(P[0], P[1], None), (ctypes.c_int64 * 3)(70000, 7, 0)
    base = [3, dt, ptr, cnt, P[2], P[3], 48, None]
    _expect(L.grad_norm, base, ({4: P[0] + 4}, SHAPE), ({4: P[1] + 12}, SHAPE), ({4: P[1] + 16}, PASSED), ({5: P[0] + 8}, SHAPE), ({4: P[3] + 4}, SHAPE))
