"""The dense block's calls whose outputs are their inputs (GPU)."""

import pytest
import torch

import sparse_matmul_ffns_amd as nm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _rand(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D", [(1, 64), (5, 1000), (33, 4096)])
def test_a_norm_in_place_returns_the_sum_that_its_gradient_reads(T, D, dtype):
    X, w, dY = _rand(T, T, D, dtype=dtype), 1 + 0.1 * _rand(1, D, dtype=torch.float32), _rand(2, T, D, dtype=dtype)
    want = nm.rms_norm(X, w)
    grads = nm.rms_norm_bwd(dY, X, w, want[2])
    x = X.clone()
    got = nm.rms_norm(x, w, Y=x)
    assert got[0] is x and all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(nm.rms_norm_bwd(dY, got[1], w, got[2]), grads))
    wide = torch.zeros(T, D + 8, dtype=dtype, device="cuda")      # a view of X
    wide[:, :D] = X
    got = nm.rms_norm(wide[:, :D], w, Y=wide[:, :D])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (wide[:, D:] == 0).all()
    want8 = nm.rms_norm_fp8(X, w, Y=torch.empty_like(X))
    x = X.clone()
    got8 = nm.rms_norm_fp8(x, w, Y=x)
    assert torch.equal(got8[0].view(torch.uint8), want8[0].view(torch.uint8))
    assert all(torch.equal(a, b) for a, b in zip(got8[1:], want8[1:]))
    # with a tensor for the sum it is taken, and X itself where nothing replaces it
    x, h = X.clone(), torch.empty_like(X)
    assert nm.rms_norm(x, w, Y=x, H=h)[1] is h and torch.equal(h, X)
    assert nm.rms_norm(X, w)[1] is X and nm.rms_norm(X, w, Y=torch.empty_like(X))[1] is X


def test_a_pass_whose_input_the_library_overwrote_is_refused():
    x, dy = _rand(0, 40, 64), _rand(1, 40, 64)
    layer = nm.DenseFFN(1 + 0.1 * _rand(2, 64), _rand(3, 96, 64), _rand(4, 64, 96), train=True)
    _, first = layer.forward(x, return_saved=True)
    _, second = layer.forward(x, return_saved=True)
    dx, _ = layer.backward(dy, first)
    nm.rms_norm(_rand(5, 40, 64), _rand(6, 64), residual=x, H=x)
    with pytest.raises(RuntimeError):
        layer.backward(dy, second)
    _, third = layer.forward(x, return_saved=True)
    nm.grad_clip([layer.W_up], 0.5)                   # a parameter
    with pytest.raises(RuntimeError):
        layer.backward(dy, third)


def test_outputs_among_the_inputs():
    """What the header allows: each output in the place of an input, and columns of one buffer beside each other."""
    for T, D in ((3, 520), (700, 4096), (600, 9000)):
        X, R, dY, dH = (_rand(i, T, D) for i in range(4))
        w = 1 + 0.1 * _rand(9, D)
        y, h, rstd = nm.rms_norm(X, w, residual=R)
        dx, dw = nm.rms_norm_bwd(dY, h, w, rstd, dH=dH)
        for into_h, into_y in ((0, 1), (1, 0), (None, 1), (0, None), (1, None)):
            xr = [X.clone(), R.clone()]
            H, Y = None if into_h is None else xr[into_h], None if into_y is None else xr[into_y]
            got = nm.rms_norm(xr[0], w, residual=xr[1], H=H, Y=Y)
            assert torch.equal(got[0], y) and torch.equal(got[1], h) and torch.equal(got[2], rstd)
            got8 = nm.rms_norm_fp8(X.clone(), w, residual=R)
            xr = [X.clone(), R.clone()]
            got = nm.rms_norm_fp8(xr[0], w, residual=xr[1], H=None if into_h is None else xr[into_h])
            assert torch.equal(got[0].view(torch.uint8), got8[0].view(torch.uint8)) and all(torch.equal(a, b) for a, b in zip(got[1:], got8[1:]))
        for k in range(3):
            a = [dY.clone(), h.clone(), dH.clone()]
            got = nm.rms_norm_bwd(a[0], a[1], w, rstd, dH=a[2], dX=a[k])
            assert got[0] is a[k] and torch.equal(got[0], dx) and torch.equal(got[1], dw)
        buf = torch.zeros(T, 4 * D, dtype=X.dtype, device="cuda")
        x, r, hh, yy = buf.split(D, 1)
        x.copy_(X), r.copy_(R)
        nm.rms_norm(x, w, residual=r, H=hh, Y=yy)
        assert torch.equal(yy, y) and torch.equal(hh, h) and torch.equal(x, X) and torch.equal(r, R)
    X, W = _rand(0, 300, 64), _rand(1, 64, 64)
    buf = torch.zeros(300, 192, dtype=X.dtype, device="cuda")
    buf[:, :64] = X
    out, pre = nm.linear_fwd(buf[:, :64], W, act="silu", residual=buf[:, :64], out=buf[:, 64:128], pre=buf[:, 128:])
    want = nm.linear_fwd(X, W, act="silu", residual=X, return_pre=True)
    assert torch.equal(out, want[0]) and torch.equal(pre, want[1]) and torch.equal(buf[:, :64], X)


def test_overlaps_are_refused():
    x, w = _rand(0, 40, 64), _rand(1, 64)
    keep = x.clone()
    with pytest.raises(nm.nmsparse.NmError):
        nm.rms_norm(x, w, H=x, Y=x)
    with pytest.raises(nm.nmsparse.NmError):
        nm.rms_norm(x[:30], w, Y=x[10:])
    with pytest.raises(nm.nmsparse.NmError):
        nm.linear_fwd(x, _rand(2, 64, 64), out=x)
    with pytest.raises(nm.nmsparse.NmError):
        nm.linear_bwd_act(x[:39], x[1:], act="silu", dZ=x.view(-1)[32:32 + 39 * 64].view(39, 64))
    flat = torch.zeros(100000, device="cuda")
    with pytest.raises(nm.nmsparse.NmError):
        nm.grad_norm([flat], norm=flat[5:6])
    assert torch.equal(x, keep) and (flat == 0).all()
