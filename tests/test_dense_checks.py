"""Refusals of the dense block's calls, in the C ABI and in the binding (CPU: nothing reaches a kernel)."""

import ctypes

import pytest
import torch

from sparse_matmul_ffns_amd import nmsparse as nm

FAKE = 1 << 20   # a non-NULL address that is never dereferenced: every call below fails validation first
OK, NULL, SHAPE, UNSUP, ALIGN = nm.NM_OK, nm.NM_ERR_NULL, nm.NM_ERR_SHAPE, nm.NM_ERR_UNSUPPORTED, nm.NM_ERR_ALIGN
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return nm.lib()


def _refuses(call, good, *bad):
    """Each of `bad` is (changes to the good arguments by position, status); the good ones are not called."""
    for change, status in bad:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert call(*args) == status, (change, status)


def test_norm(L):
    # dt, X, ldx, residual, ldr, wdt, w, eps, T, D, H, ldh, Y, ldy, rstd, stream
    good = [1, FAKE, 16, FAKE, 16, 1, FAKE, 1e-5, 4, 16, FAKE, 16, FAKE, 16, FAKE, None]
    _refuses(L.rms_norm, good, ({1: None}, NULL), ({6: None}, NULL), ({12: None}, NULL), ({0: 2}, UNSUP), ({5: 2}, UNSUP),
             ({7: 0.0}, UNSUP), ({7: -1.0}, UNSUP), ({7: NAN}, UNSUP), ({7: INF}, UNSUP), ({8: 0}, SHAPE), ({8: 1 << 31}, SHAPE),
             ({9: 0}, SHAPE), ({9: 17}, SHAPE), ({2: 15}, SHAPE), ({4: 15}, SHAPE), ({11: 15}, SHAPE), ({13: 15}, SHAPE),
             ({9: 16385, 2: 16385, 4: 16385, 11: 16385, 13: 16385}, UNSUP), ({1: FAKE + 1}, ALIGN), ({3: FAKE + 1}, ALIGN),
             ({6: FAKE + 1}, ALIGN), ({10: FAKE + 1}, ALIGN), ({12: FAKE + 1}, ALIGN), ({14: FAKE + 2}, ALIGN),
             ({0: 0, 1: FAKE + 2}, ALIGN))
    # dt, X, ldx, residual, ldr, wdt, w, eps, T, D, fmt, Q, ldq, S, lds, H, ldh, Y, ldy, rstd, stream
    good = [1, FAKE, 16, FAKE, 16, 1, FAKE, 1e-5, 4, 16, 0, FAKE, 128, FAKE, 4, FAKE, 16, None, 0, FAKE, None]
    _refuses(L.rms_norm_fp8, good, ({11: None}, NULL), ({13: None}, NULL), ({1: None}, NULL), ({10: 2}, UNSUP),
             ({12: 127}, SHAPE), ({14: 3}, SHAPE), ({13: FAKE + 2}, ALIGN), ({17: FAKE, 18: 15}, SHAPE), ({7: 0.0}, UNSUP))
    # dt, dY, lddy, H, ldh, wdt, w, rstd, dH, lddh, T, D, dX, lddx, dw, work, work_bytes, stream
    need = ctypes.c_int64()
    assert L.rms_norm_bwd_work_bytes(4, 2000, ctypes.byref(need)) == OK and need.value >= 4 * 2000 * 4
    assert L.rms_norm_bwd_work_bytes(1, 2000, ctypes.byref(need)) == OK and need.value == 0
    assert L.rms_norm_bwd_work_bytes(0, 16, ctypes.byref(need)) == SHAPE
    assert L.rms_norm_bwd_work_bytes(4, 16385, ctypes.byref(need)) == UNSUP
    assert L.rms_norm_bwd_work_bytes(4, 16, None) == NULL
    good = [1, FAKE, 2000, FAKE, 2000, 0, FAKE, FAKE, FAKE, 2000, 4, 2000, FAKE, 2000, FAKE, FAKE, 1 << 20, None]
    _refuses(L.rms_norm_bwd, good, *[({i: None}, NULL) for i in (1, 3, 6, 7, 12, 14, 15)], ({0: 3}, UNSUP), ({5: 3}, UNSUP),
             *[({i: 1999}, SHAPE) for i in (2, 4, 9, 13)], ({16: 4 * 2000 * 4 - 1}, SHAPE), ({10: 0}, SHAPE),
             *[({i: FAKE + 1}, ALIGN) for i in (1, 3, 6, 7, 8, 12, 14, 15)])


def test_linear(L):
    # dt, X, ldx, W, ldw, bdt, bias, act, residual, ldr, M, N, K, out, Y, ldy, pre, ldp, work, work_bytes, stream
    good = [1, FAKE, 32, FAKE, 32, 1, FAKE, 1, FAKE, 16, 4, 16, 32, 1, FAKE, 16, FAKE, 16, FAKE, 64, None]
    _refuses(L.linear_fwd, good, *[({i: None}, NULL) for i in (1, 3, 14)], ({0: 0}, UNSUP), ({5: 2}, UNSUP), ({7: 4}, UNSUP),
             ({7: -1}, UNSUP), ({13: 2}, UNSUP), *[({i: 0}, SHAPE) for i in (10, 11, 12)], ({10: 1 << 31}, SHAPE),
             *[({i: 31}, SHAPE) for i in (2, 4)], *[({i: 15}, SHAPE) for i in (9, 15, 17)],
             *[({i: FAKE + 1}, ALIGN) for i in (1, 3, 6, 8, 14, 16)], ({5: 0, 6: FAKE + 2}, ALIGN), ({13: 0, 14: FAKE + 2}, ALIGN),
             ({18: FAKE + 8}, ALIGN))
    # dt, dY, lddy, pre, ldp, act, M, N, dZ, lddz, db, work, work_bytes, stream
    good = [1, FAKE, 16, FAKE, 16, 2, 4000, 16, FAKE, 16, FAKE, FAKE, 1 << 20, None]
    _refuses(L.linear_bwd_act, good, ({1: None}, NULL), ({3: None}, NULL), ({8: None, 10: None}, NULL), ({11: None}, NULL),
             ({0: 0}, UNSUP), ({5: 9}, UNSUP), ({6: 0}, SHAPE), ({7: 0}, SHAPE), ({2: 15}, SHAPE), ({4: 15}, SHAPE), ({9: 15}, SHAPE),
             ({12: 0}, SHAPE), ({1: FAKE + 1}, ALIGN), ({3: FAKE + 1}, ALIGN), ({8: FAKE + 1}, ALIGN), ({10: FAKE + 2}, ALIGN),
             ({11: FAKE + 2}, ALIGN))
    need = ctypes.c_int64()
    assert L.linear_bwd_act_work_bytes(4000, 16, ctypes.byref(need)) == OK and need.value > 0
    assert L.linear_bwd_act_work_bytes(1, 16, ctypes.byref(need)) == OK and need.value == 0
    assert L.linear_bwd_act_work_bytes(1, 0, ctypes.byref(need)) == SHAPE
    assert L.linear_bwd_act_work_bytes(1, 1, None) == NULL
    # dt, dZ, lddz, W, ldw, pre, ldp, act, M, N, K, out, dX, lddx, work, work_bytes, stream
    good = [1, FAKE, 16, FAKE, 32, FAKE, 32, 1, 4, 16, 32, 1, FAKE, 32, None, 0, None]
    _refuses(L.linear_bwd_x, good, *[({i: None}, NULL) for i in (1, 3, 5, 12)], ({0: 0}, UNSUP), ({7: 4}, UNSUP), ({11: 2}, UNSUP),
             ({2: 15}, SHAPE), ({4: 31}, SHAPE), ({6: 31}, SHAPE), ({13: 31}, SHAPE), *[({i: 0}, SHAPE) for i in (8, 9, 10)],
             *[({i: FAKE + 1}, ALIGN) for i in (1, 3, 5, 12)], ({14: FAKE + 8}, ALIGN))
    # dt, dZ, lddz, X, ldx, M, N, K, accumulate, out, dW, lddw, work, work_bytes, stream
    good = [1, FAKE, 16, FAKE, 32, 4, 16, 32, 0, 0, FAKE, 32, None, 0, None]
    _refuses(L.linear_bwd_w, good, *[({i: None}, NULL) for i in (1, 3, 10)], ({0: 0}, UNSUP), ({9: 2}, UNSUP), ({8: 1, 9: 1}, UNSUP),
             ({2: 15}, SHAPE), ({4: 31}, SHAPE), ({11: 31}, SHAPE), *[({i: 0}, SHAPE) for i in (5, 6, 7)],
             ({1: FAKE + 1}, ALIGN), ({3: FAKE + 1}, ALIGN), ({10: FAKE + 2}, ALIGN), ({12: FAKE + 8}, ALIGN))
    # which, M, N, K, aligned, bytes: parts where tiles are few and the reduction long, copies where rows are not aligned
    need = ctypes.c_int64()
    for which, sizes, al, some in ((0, (512, 2048, 8192), 1, True), (0, (1, 2048, 8192), 1, False), (0, (8192, 16384, 4096), 1, False),
                                   (1, (32, 8192, 2048), 1, True), (2, (8192, 256, 256), 1, True), (2, (64, 4096, 4096), 1, False),
                                   (0, (8192, 16384, 4096), 0, True), (0, (1, 2048, 8192), 0, False), (0, (8192, 16384, 4095), 1, True),
                                   (1, (4096, 4096, 4095), 1, True), (2, (4095, 4096, 4096), 1, False), (0, (8, 8, 8), 0, False)):
        assert L.linear_work_bytes(which, *sizes, al, ctypes.byref(need)) == OK and (need.value > 0) == some, (which, sizes)
    assert L.linear_work_bytes(0, 4096, 4104, 4095, 1, ctypes.byref(need)) == OK
    assert need.value == (4096 + 4104) * 4096 * 2
    assert L.linear_work_bytes(3, 1, 1, 1, 1, ctypes.byref(need)) == UNSUP
    assert L.linear_work_bytes(0, 0, 1, 1, 1, ctypes.byref(need)) == SHAPE and L.linear_work_bytes(0, 1, 1, 1, 1, None) == NULL


def _lists(ptrs, counts, dts):
    n = len(ptrs)
    return (ctypes.c_int * n)(*dts), (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*counts)


def test_grads(L):
    need = ctypes.c_int64()
    assert L.grad_work_bytes(2, (ctypes.c_int64 * 2)(16384, 16385), ctypes.byref(need)) == OK and need.value == 0
    assert L.grad_work_bytes(2, (ctypes.c_int64 * 2)(65536, 1), ctypes.byref(need)) == OK and need.value == 5 * 8
    assert L.grad_work_bytes(200, (ctypes.c_int64 * 200)(*[1] * 200), ctypes.byref(need)) == OK and need.value == 200 * 8
    assert L.grad_work_bytes(2, (ctypes.c_int64 * 2)(0, 0), ctypes.byref(need)) == OK and need.value == 0
    assert L.grad_work_bytes(1, (ctypes.c_int64 * 1)(1 << 40), ctypes.byref(need)) == OK and need.value == 1024 * 8
    assert L.grad_work_bytes(1, (ctypes.c_int64 * 1)(-1), ctypes.byref(need)) == SHAPE
    assert L.grad_work_bytes(0, (ctypes.c_int64 * 1)(1), ctypes.byref(need)) == SHAPE
    assert L.grad_work_bytes(1, None, ctypes.byref(need)) == NULL
    W = 1 << 30
    dt, ptr, cnt = _lists([FAKE, FAKE + 400000], [70000, 7], [0, 1])
    good = [2, dt, ptr, cnt, W, W + 4096, 1 << 16, None]      # n, dt, grads, counts, norm, work, work_bytes, stream
    _refuses(L.grad_norm, good, ({0: 0}, SHAPE), ({0: 65537}, SHAPE), *[({i: None}, NULL) for i in (1, 2, 3, 4, 5)], ({6: 39}, SHAPE),
             ({4: W + 2}, ALIGN), ({5: W + 4100}, ALIGN), ({1: _lists([1, 1], [1, 1], [0, 2])[0]}, UNSUP),
             ({2: _lists([FAKE, 0], [1, 1], [0, 0])[1]}, NULL), ({2: _lists([FAKE + 2, FAKE], [1, 1], [0, 0])[1]}, ALIGN),
             ({3: _lists([1, 1], [1, -1], [0, 0])[2]}, SHAPE))
    # n, dt, grads, counts, max_norm, have_norm, norm, odt, out, work, work_bytes, stream
    good = [2, dt, ptr, cnt, 1.0, 0, W, dt, ptr, W + 4096, 1 << 16, None]
    at = lambda *p: _lists(p, [1] * len(p), [0] * len(p))[1]
    _refuses(L.grad_clip, good, ({4: NAN}, UNSUP), ({4: -1.0}, UNSUP), ({7: None}, NULL), ({8: None}, NULL), ({9: None}, NULL),
             ({10: 8}, SHAPE), ({8: at(FAKE, 0)}, NULL), ({8: at(FAKE + 1, FAKE + 4096)}, ALIGN),
             ({7: _lists([1, 1], [1, 1], [0, 5])[0]}, UNSUP),
             # outputs that meet each other, another's gradient, their own gradient shifted or in another type
             ({8: at(FAKE + 8192, FAKE + 8192)}, SHAPE), ({8: at(FAKE + 4096 + 4, FAKE + 16384)}, SHAPE),
             ({8: at(FAKE + 4, FAKE + 4096)}, SHAPE), ({7: _lists([1, 1], [1, 1], [1, 1])[0]}, SHAPE),
             ({8: at(FAKE + 8192, FAKE + 396)}, SHAPE),
             # the norm or the work memory inside a tensor
             ({6: FAKE + 8}, SHAPE), ({9: FAKE + 8}, SHAPE))
    # the same gradient twice, in place
    dt2, ptr2, cnt2 = _lists([FAKE, FAKE], [4, 4], [0, 0])
    assert L.grad_clip(2, dt2, ptr2, cnt2, 1.0, 0, W, dt2, ptr2, W + 4096, 1 << 16, None) == SHAPE


class Library:
    def __getattr__(self, name):
        def reached(*args):
            raise AssertionError("the call reached the library")
        return reached


@pytest.fixture
def no_device(monkeypatch):
    monkeypatch.setattr(nm, "_here", lambda *ts: None)
    monkeypatch.setattr(nm, "_here_all", lambda ts: None)
    monkeypatch.setattr(nm, "_stream", lambda: None)
    monkeypatch.setattr(nm, "lib", Library)
    monkeypatch.setattr(nm, "_norm_work_bytes", lambda T, D: 0)
    monkeypatch.setattr(nm, "_act_work_bytes", lambda M, N: 0)
    monkeypatch.setattr(nm, "_linear_work_bytes", lambda call, M, N, K, aligned: 0)


def _b(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


CALLS = {
    "rms_norm": dict(X=_b(4, 16), w=torch.ones(16), residual=_b(4, 16), H=_b(4, 16), Y=_b(4, 16), rstd=torch.ones(4)),
    "rms_norm_fp8": dict(X=_b(4, 200), w=torch.ones(200), residual=_b(4, 200), H=_b(4, 200), Y=_b(4, 200),
                         Q=torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn), S=torch.ones(2, 4)),
    "rms_norm_bwd": dict(dY=_b(4, 16), H=_b(4, 16), w=torch.ones(16), rstd=torch.ones(4), dH=_b(4, 16), dX=_b(4, 16),
                         dw=torch.ones(16)),
    "linear_fwd": dict(X=_b(4, 16), W=_b(8, 16), bias=_b(8), residual=_b(4, 8), out=_b(4, 8), pre=_b(4, 8)),
    "linear_bwd_act": dict(dY=_b(4, 8), pre=_b(4, 8), act="silu", dZ=_b(4, 8), db=torch.ones(8)),
    "linear_bwd_x": dict(dZ=_b(4, 8), W=_b(8, 16), pre=_b(4, 16), act="relu", out=_b(4, 16)),
    "linear_bwd_w": dict(dZ=_b(4, 8), X=_b(4, 16), out=torch.zeros(8, 16)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_binding_refuses_other_shapes_and_types(no_device, name):
    call, good = getattr(nm, name), CALLS[name]
    with pytest.raises(AssertionError):
        call(**good)
    for key, t in good.items():
        if not torch.is_tensor(t):
            continue
        others = [t.reshape(1, *t.shape), torch.zeros(tuple(s + 1 for s in t.shape), dtype=t.dtype)]
        if t.dim() == 2:
            others += [t.reshape(-1).contiguous(), torch.zeros(t.shape[1], t.shape[0], dtype=t.dtype).t()]
        for other in others:
            with pytest.raises((ValueError, TypeError)):
                call(**dict(good, **{key: other}))
        with pytest.raises((ValueError, TypeError)):
            call(**dict(good, **{key: t.to(torch.float64)}))


def test_binding_refuses_lists_and_options(no_device, monkeypatch):
    g = [torch.zeros(3, 4), _b(5)]
    with pytest.raises(AssertionError):
        nm.grad_norm(g)
    for bad in ([], [torch.zeros(4, 4)[:, :2]], [torch.zeros(3, dtype=torch.float16)], [None, g[0]],
                [torch.zeros(4).expand(3, 4)]):
        with pytest.raises((ValueError, TypeError)):
            nm.grad_norm(bad)
        with pytest.raises((ValueError, TypeError)):
            nm.grad_clip(bad, 1.0)
    for out in ([g[0]], [g[1], g[0]], [torch.zeros(4, 3), _b(5)], [torch.zeros(4, 3).t(), _b(5)]):
        with pytest.raises(ValueError):
            nm.grad_clip(g, 1.0, out=out)
    for norm in (torch.zeros(2), torch.zeros(()), torch.zeros(1, dtype=torch.float64)):
        with pytest.raises((ValueError, TypeError)):
            nm.grad_clip(g, 1.0, norm=norm)
    with pytest.raises(ValueError):
        nm.linear_fwd(_b(4, 16), _b(8, 16), act="gelu")
    with pytest.raises(ValueError):
        nm.linear_bwd_act(_b(4, 8), act="silu")
    with pytest.raises(ValueError):
        nm.linear_bwd_x(_b(4, 8), _b(8, 16), act="silu")
    with pytest.raises(ValueError):
        nm.linear_bwd_w(_b(4, 8), _b(4, 16), accumulate=True)
    with pytest.raises(ValueError):
        nm.rms_norm_bwd(_b(4, 8), _b(4, 8), torch.ones(8), torch.ones(4), work="more")


def test_binding_refuses_another_device(monkeypatch):
    class On:
        is_cuda = True

        def __init__(self, i):
            self.i = i

        def get_device(self):
            return self.i

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    nm._here(On(1), None)
    with pytest.raises(ValueError):
        nm._here(On(1), On(0))
    with pytest.raises(ValueError):
        nm._here(torch.zeros(1))
