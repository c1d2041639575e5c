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
