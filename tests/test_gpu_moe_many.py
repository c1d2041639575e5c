"""More tokens or rows than the work-items of one launch hold (GPU): the runtime takes a grid of 2^32
work-items or more modulo 2^32 without an error, so a call in one launch would leave all but the last few
rows as they were.  Values are exact, every row is compared.
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


def _i32(T, k=1):
    return torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)


def test_combine():
    T, D = (1 << 26) + 5, 8                                   # 64 work-items a token
    O = torch.arange(1, 5, dtype=torch.bfloat16, device="cuda").view(4, 1).repeat(1, D)
    pos = _i32(T) % 4
    w = (1.0 + (_i32(T) % 3)).float()
    for weights in (None, w):
        Y = torch.full((T, D), 99.0, dtype=torch.bfloat16, device="cuda")
        nm.moe_combine(O, pos, weights, out=Y)
        want = (pos + 1).bfloat16() * (1 if weights is None else w.bfloat16())
        assert bool((Y == want).all())


@pytest.mark.parametrize("T,extra", [((1 << 24) + 5, 0), (3, (1 << 26) + 37)])
def test_combine_gradients(T, extra):
    """Many tokens, and few tokens with many rows of no slot: 256 work-items a token or 16 rows."""
    D, rows = 8, T + extra
    dY = (_i32(T) % 5 - 2).bfloat16().repeat(1, D)
    pos = rows - 1 - _i32(T)                                  # the rows in descending order
    src = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    src[pos.view(-1).long()] = _i32(T).view(-1)
    w = (1.0 + (_i32(T) % 3)).float()
    O = torch.ones(1, D, dtype=torch.bfloat16, device="cuda").expand(rows, D).contiguous()
    dO = torch.full((rows, D), 99.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, 1), 99.0, device="cuda")
    nm.moe_combine_bwd(dY, O, src, pos, w, dO=dO, dweights=dw)
    assert bool((dw == D * dY[:, :1].float()).all())
    assert bool((dO[pos.view(-1).long()] == dY * w.bfloat16()).all())
    assert not dO[:extra].any()


def test_route_and_its_gradient():
    T, E, k = (1 << 28) + 7, 8, 1                             # 16 work-items a token
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    best = _i32(T) % E
    logits.scatter_(1, best.long(), 1.0)
    ids, w = nm.moe_route(logits, k, ids=torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
                          weights=torch.full((T, k), 99.0, device="cuda"))
    assert torch.equal(ids, best) and bool((w == 1.0).all())
    del w
    # a plain sigmoid's gradient: one place a token, w dw (1 - s) with w = 0.5
    half = torch.full((T, k), 0.5, device="cuda")
    logits.zero_()
    dl = torch.full((T, E), 99.0, dtype=torch.bfloat16, device="cuda")
    nm.moe_route_bwd(logits, ids, half, half * 8, score="sigmoid", renorm=False, dlogits=dl)
    assert bool((dl.sum(1, keepdim=True) == 1.0).all())
    assert bool((torch.gather(dl, 1, best.long()) == 1.0).all())


@pytest.mark.parametrize("gather", [False, True])
def test_quantize(gather):
    R, K = (1 << 28) + 9, 1                                   # 16 work-items a row
    X = (_i32(R) % 7 + 1).bfloat16()
    src = (R - 1 - _i32(R)).view(-1) if gather else None
    gate = X if not gather else (_i32(R) % 2).bfloat16()
    q, s = nm.fp8_quantize(X, src=src, gate=gate)
    want = X.view(-1).flip(0) * gate.view(-1) if gather else X.view(-1)
    del X, gate, src
    got = q[:, 0].contiguous().bfloat16() * s[0].bfloat16()
    assert torch.equal(got, want)
    for r in (0, 1 << 24, R - 1):
        assert not q[r, 1:].view(torch.uint8).any()


def test_product():
    M = (1 << 30) + 70                                        # four work-items a row: unaligned rows
    a = (torch.arange(M, dtype=torch.int32, device="cuda") % 7 + 1).view(M, 1)
    A = a.to(torch.float8_e4m3fn)
    C = nm.fp8_gemm_nt(A, torch.ones(1, M, device="cuda"), torch.ones(1, 1, device="cuda").to(torch.float8_e4m3fn),
                       torch.ones(1, 1, device="cuda"), out=torch.full((M, 1), 99.0, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(C, a.bfloat16())
