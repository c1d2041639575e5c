"""The dense block's operators where offsets pass 32 bits: rows and strides of several GB, and more elements than fit 31 bits.
Products of small integers are exact; rows of a norm do not depend on each other, so the last rows of a large call are
those of a small one, bit for bit.
"""

import pytest
import torch

import sparse_matmul_ffns_amd as nm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def _wide(R, C, ld, dtype=torch.bfloat16, fill=0.0):
    return torch.full((R, ld), fill, device="cuda", dtype=dtype)[:, :C]


def _ints(g, t):
    return t.copy_(torch.randint(-3, 4, t.shape, generator=g, device="cuda"))


# rows, the stride of all matrices: aligned (the tiles), not aligned (copies, and the general kernel without work), and more than
# the tiles' descriptors hold
@pytest.mark.parametrize("M,ld", [(66000, 40000), (66000, 40001), (1100, (1 << 21) + 8), (600, (1 << 22) + 8)])
def test_products(M, ld):
    g = torch.Generator(device="cuda").manual_seed(M + ld)
    N, K = 264, 136
    X, D, Y = _ints(g, _wide(M, K, ld)), _ints(g, _wide(M, N, ld)), _wide(M, N, ld, fill=5.0)
    W = _ints(g, torch.empty(N, K, device="cuda", dtype=torch.bfloat16))
    R, P = _ints(g, _wide(M, N, ld)), _wide(M, N, ld)
    z = X.double() @ W.double().t()
    for work in ("auto", None):
        nm.linear_fwd(X, W, residual=R, out=Y, pre=P, work=work)
        assert torch.equal(P, z.bfloat16()) and torch.equal(Y, (z + R.double()).bfloat16())
        dX = _wide(M, K, ld)
        nm.linear_bwd_x(D, W, pre=X, act="relu", out=dX, work=work)
        dx = D.double() @ W.double()
        assert torch.equal(dX, torch.where(X > 0, dx, torch.zeros_like(dx)).bfloat16())
        del dX
        # sums over 66000 rows of products up to 9 stay below 2^24
        assert torch.equal(nm.linear_bwd_w(D, X, work=work), (D.double().t() @ X.double()).float())
    assert bool((Y._base[:, N:N + 8] == 5).all())


def test_a_wide_weight():
    """W and dW of 5 GB: 20000 rows of 131072."""
    g = torch.Generator(device="cuda").manual_seed(1)
    M, N, K = 8, 20000, 131072
    W = torch.zeros(N, K, device="cuda", dtype=torch.bfloat16)
    W[N - 300:] = torch.randint(-3, 4, (300, K), generator=g, device="cuda")
    X = _ints(g, torch.empty(M, K, device="cuda", dtype=torch.bfloat16))
    D = _ints(g, torch.empty(M, N, device="cuda", dtype=torch.bfloat16))
    assert torch.equal(nm.linear_fwd(X, W), torch.cat([torch.zeros(M, N - 300, device="cuda"), (X.double() @ W[N - 300:].double().t()).float()],
                                                      1).bfloat16())
    assert torch.equal(nm.linear_bwd_x(D, W), (D[:, N - 300:].double() @ W[N - 300:].double()).bfloat16())
    dW = nm.linear_bwd_w(D, X)
    for r in (0, N // 2, N - 300):
        assert torch.equal(dW[r:r + 300], (D[:, r:r + 300].double().t() @ X.double()).float())


@pytest.mark.parametrize("M,K", [(3, 8), (3, 5), (40, 16), (40, 11)])
@pytest.mark.parametrize("N", [(1 << 21) + 70, (1 << 22) + 5001])
def test_many_columns(M, N, K):
    """More columns than a launch takes at once, in each product."""
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    X, W, R = (_ints(g, torch.empty(s, device="cuda", dtype=torch.bfloat16)) for s in ((M, K), (N, K), (M, N)))
    b = _ints(g, torch.empty(N, device="cuda", dtype=torch.bfloat16))
    z = X.double() @ W.double().t() + b.double()
    for work in ("auto", None):
        Y, P = nm.linear_fwd(X, W, bias=b, act="relu", residual=R, return_pre=True, work=work)
        assert torch.equal(P, z.bfloat16()) and torch.equal(Y, (z.clamp(min=0) + R.double()).bfloat16())
        D, V = X, W.t().contiguous()                      # dX [M, N] of D [M, K] and a weight [K, N]
        dx = D.double() @ V.double()
        assert torch.equal(nm.linear_bwd_x(D, V, pre=R, act="relu", work=work), torch.where(R > 0, dx, torch.zeros_like(dx)).bfloat16())
        D = X.t().contiguous()                            # dW [M, N] of D [K, M] and X [K, N]
        dW = torch.ones(M, N, device="cuda")
        nm.linear_bwd_w(D, V, out=dW, accumulate=True, work=work)
        assert torch.equal(dW, (1 + dx).float())


def test_norm_of_many_rows():
    g = torch.Generator(device="cuda").manual_seed(2)
    T, D, n = 330000, 8192, 40
    X = torch.randn(D, generator=g, device="cuda").bfloat16().expand(T, D).contiguous()
    X[T - n:] = torch.randn(n, D, generator=g, device="cuda")
    w = torch.randn(D, generator=g, device="cuda").bfloat16()
    H, r = torch.empty_like(X), torch.empty(T, device="cuda")
    Y, _, _ = nm.rms_norm(X, w, residual=X, H=H, rstd=r)
    few = X[T - n:].clone()
    h, q = torch.empty_like(few), torch.empty(n, device="cuda")
    y, _, _ = nm.rms_norm(few, w, residual=few, H=h, rstd=q)
    assert torch.equal(Y[T - n:], y) and torch.equal(H[T - n:], h) and torch.equal(r[T - n:], q)
    assert torch.equal(Y[:1], Y[T - n - 1:T - n])
    y8, s8, _, _ = nm.rms_norm_fp8(few, w)
    Y8, S8, _, _ = nm.rms_norm_fp8(X, w)
    assert torch.equal(Y8[T - n:].view(torch.uint8), y8.view(torch.uint8)) and torch.equal(S8[:, T - n:], s8)
    dY = torch.zeros_like(X)
    dY[T - n:] = torch.randn(n, D, generator=g, device="cuda")
    dX, dw = nm.rms_norm_bwd(dY, H, w, r)
    dx, dw1 = nm.rms_norm_bwd(dY[T - n:].clone(), h, w, q)
    assert torch.equal(dX[T - n:], dx) and not bool(dX[:T - n].any())
    # the same n terms in another order on each side: n steps each, of half a step of fp32 of their magnitudes
    mag = (dY[T - n:].double() * h.double() * q.double()[:, None]).abs().sum(0)
    assert bool(((dw.double() - dw1.double()).abs() <= (2 * n + 8) * 2 ** -24 * mag).all())


def test_norm_of_wide_rows_past_one_launch():
    """4194307 rows of 8200 (69 GB, in place): at 1024 work-items a row, more than 2^32 of them."""
    g = torch.Generator(device="cuda").manual_seed(4)
    T, D, n = (1 << 22) + 3, 8200, 4096
    base = torch.randn(n, D, generator=g, device="cuda").bfloat16()
    w = torch.randn(D, generator=g, device="cuda").bfloat16()
    X, rstd = torch.empty(T, D, device="cuda", dtype=torch.bfloat16), torch.zeros(T, device="cuda")
    for r in range(0, T, n):
        X[r:r + n] = base[:T - r]
    want, _, r0 = nm.rms_norm(base, w)
    nm.rms_norm(X, w, Y=X, rstd=rstd)
    for r in range(0, T, n):
        m = min(n, T - r)
        assert torch.equal(X[r:r + m], want[:m]) and torch.equal(rstd[r:r + m], r0[:m]), r


def test_act_gradient_of_many_rows():
    g = torch.Generator(device="cuda").manual_seed(3)
    M, N, n = 290000, 8192, 24
    dY = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    dY[M - n:] = torch.randint(-3, 4, (n, N), generator=g, device="cuda")
    pre = torch.ones(M, N, device="cuda", dtype=torch.bfloat16)
    pre[M - n:] = torch.randint(-3, 4, (n, N), generator=g, device="cuda")
    db = torch.empty(N, device="cuda")
    dZ = nm.linear_bwd_act(dY, pre, act="relu", db=db)
    want = torch.where(pre[M - n:] > 0, dY[M - n:], torch.zeros_like(dY[M - n:]))
    dZ = dZ[0] if isinstance(dZ, tuple) else dZ
    assert torch.equal(dZ[M - n:], want) and not bool(dZ[:M - n].any()) and torch.equal(db, want.float().sum(0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_clip_of_more_elements_than_31_bits(dtype):
    n = (1 << 31) + 5
    a = torch.zeros(n, device="cuda", dtype=dtype)
    at = torch.tensor([0, 1 << 30, (1 << 31) - 1, 1 << 31, n - 1], device="cuda")
    a[at] = torch.tensor([2.0, -4.0, 4.0, 8.0, 0.0], device="cuda", dtype=dtype)     # squares 4 + 16 + 16 + 64
    b = torch.full((21,), 2.0, device="cuda")                                        # and 84
    out = [torch.empty_like(a), torch.empty_like(b)]
    norm = nm.grad_clip([a, b], 1.0, out=out)
    assert float(norm) == float(torch.tensor(184.0, dtype=torch.float64).sqrt().float())
    f = 1 / 184.0 ** 0.5      # the norm, the factor and the product are rounded: 4 halves of a step of fp32, and bf16's
    tol = 2.0 ** -22 + (2.0 ** -8 if dtype == torch.bfloat16 else 0)
    assert bool(((out[0][at].double() - a[at].double() * f).abs() <= a[at].double().abs() * f * tol).all())
    assert int(torch.count_nonzero(out[0])) == 4 and bool((out[1] == out[1][0]).all())
