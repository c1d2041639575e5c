"""The mixture-of-experts calls on operands whose offsets pass 32 bits (GPU): the last rows and the last
expert of arrays of more than 4 GiB, against torch on those rows alone.  Small integers, so every sum is
exact.
"""

import pytest
import torch

import sparse_matmul_ffns_amd as nm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _ints(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda").float()


@pytest.mark.parametrize("rows", [8, 300])
def test_last_expert_of_a_large_weight(rows):
    E, N, K = 160, 8192, 4096                                  # 5.4 GB of weights
    B = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    b = _ints(N, K, seed=1)
    B[E - 1] = b.to(torch.float8_e4m3fn)
    a = _ints(rows, K, seed=2)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = rows
    ones = lambda *s: torch.ones(*s, device="cuda")
    C = nm.fp8_gemm_nt_grouped(a.to(torch.float8_e4m3fn), ones(K // 128, rows), B, ones(E, N // 128, K // 128), off,
                               out_dtype=torch.float32)
    assert torch.equal(C, (a.double() @ b.double().t()).float())


def test_last_rows_of_large_operands():
    M, K, N = 1 << 20, 4224, 256                               # A 4.4 GB, C 1.1 GB
    A = torch.zeros(M, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    a, b = _ints(300, K, seed=3), _ints(N, K, seed=4)
    A[M - 300:] = a.to(torch.float8_e4m3fn)
    sa = torch.ones(K // 128, M, device="cuda")
    sb = torch.ones(N // 128, K // 128, device="cuda")
    C = nm.fp8_gemm_nt(A, sa, b.to(torch.float8_e4m3fn), sb, out_dtype=torch.float32)
    assert torch.equal(C[M - 300:], (a.double() @ b.double().t()).float())
    assert not C[:M - 300].any()
    del A, sa, C
    X = torch.zeros(M, 2304, dtype=torch.bfloat16, device="cuda")   # 4.8 GB
    x = _ints(256, 2304, seed=5).bfloat16()
    X[M - 256:] = x
    src = torch.arange(M - 256, M, dtype=torch.int32, device="cuda")
    for call in (nm.fp8_quantize, nm.fp8_quantize_t):
        got, want = call(X, src=src), call(x)
        assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
    q, s = nm.fp8_quantize(X)
    want = nm.fp8_quantize(x)
    assert torch.equal(q[M - 256:].view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(s[:, M - 256:], want[1])
    pos = torch.tensor([[M - 1, 0, M - 256]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[2.0, 1.0, 3.0]], device="cuda")
    y = nm.moe_combine(X, pos, w)
    assert torch.equal(y[0].float(), 2 * x[255].float() + 3 * x[0].float())
