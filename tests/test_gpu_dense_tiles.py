"""The dense products' large tiles: products of small integers, whose sums are exact in fp32 in every order, at
sizes that take the 256 x 256 tiles (hundreds of tiles, ragged at each edge), bit for bit against 64-bit products on
the GPU; and the same with rows that start elsewhere and outputs between guards.
"""

import pytest
import torch

import sparse_matmul_ffns_amd as nm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _ints(g, R, C, pad=0):
    t = torch.randint(-3, 4, (R, C + pad), generator=g, device="cuda").bfloat16()
    if pad:
        t[:, C:] = float("nan")
    return t[:, :C]


def _guarded(R, C, dtype, pad):
    flat = torch.full((R, C + pad), 77.0, device="cuda", dtype=dtype)
    return flat[:, :C], flat[:, C:]


CASES = [(4096, 4104, 8, 0), (4096, 4104, 32, 8), (4100, 4096, 40, 0), (4097, 4232, 64, 0), (3850, 4352, 96, 16), (4096, 4096, 128, 0),
         (4103, 4120, 168, 8), (8192, 2056, 200, 0), (2049, 8200, 320, 24)]


@pytest.mark.parametrize("M,N,K,pad", CASES)
def test_forward(M, N, K, pad):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    X, W, R, b = _ints(g, M, K, pad), _ints(g, N, K, pad), _ints(g, M, N, pad), _ints(g, 1, N)[0]
    z = X.double() @ W.double().t()
    for out in (torch.bfloat16, torch.float32):
        Y, guard = _guarded(M, N, out, pad + 8)
        assert torch.equal(nm.linear_fwd(X, W, out=Y), z.to(out)) and bool((guard == 77).all())
        P, pguard = _guarded(M, N, torch.bfloat16, pad + 16)
        nm.linear_fwd(X, W, bias=b, act="relu", residual=R, out=Y, pre=P)
        zb = z + b.double()
        assert torch.equal(P, zb.bfloat16()) and torch.equal(Y, (zb.clamp(min=0) + R.double()).to(out))
        assert bool((guard == 77).all()) and bool((pguard == 77).all())


@pytest.mark.parametrize("M,N,K,pad", CASES)
def test_gradients(M, N, K, pad):
    """dX [M, N] = dZ [M, K] W [K, N] and dW [M, N] = dZ [K, M]^T X [K, N]: results of the forward's sizes."""
    g = torch.Generator(device="cuda").manual_seed(M + N + K + 1)
    D, W, P = _ints(g, M, K, pad), _ints(g, K, N, pad), _ints(g, M, N, pad)
    want = D.double() @ W.double()
    for out in (torch.bfloat16, torch.float32):
        Y, guard = _guarded(M, N, out, pad + 8)
        nm.linear_bwd_x(D, W, out=Y)
        assert torch.equal(Y, want.to(out)) and bool((guard == 77).all())
        nm.linear_bwd_x(D, W, pre=P, act="relu", out=Y)
        assert torch.equal(Y, torch.where(P > 0, want, torch.zeros_like(want)).to(out)) and bool((guard == 77).all())
    M8 = M // 8 * 8
    D, X = _ints(g, K + 3, M8, pad), _ints(g, K + 3, N, pad)       # any number of rows
    want = D.double().t() @ X.double()
    Y, guard = _guarded(M8, N, torch.float32, pad + 8)
    nm.linear_bwd_w(D, X, out=Y)
    assert torch.equal(Y, want.float())
    nm.linear_bwd_w(D, X, out=Y, accumulate=True)
    assert torch.equal(Y, 2 * want.float()) and bool((guard == 77).all())


def test_repeats_are_equal():
    """Ordinary values: the same call gives the same bits, again and next to other work."""
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(4100, 520, generator=g, device="cuda").bfloat16()
    W = torch.randn(4104, 520, generator=g, device="cuda").bfloat16()
    D = torch.randn(4100, 4104, generator=g, device="cuda").bfloat16()
    first = None
    side = torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(side):
            nm.linear_bwd_w(D, X)
        got = [nm.linear_fwd(X, W, act="silu", residual=D), nm.linear_bwd_x(D, W), nm.linear_bwd_w(D, X)]
        torch.cuda.synchronize()
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
