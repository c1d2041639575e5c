"""Scales far from 1 in the 8-bit products (GPU).

All operands are 448, so a block's sum is 128 * 448^2 = 49 * 2^19, and with the scales' product a power of
two every result is exact in fp32 and in bf16: C = blocks * 49 * 2^19 * sa * sb.  A scale of 2^110 times the
sum alone passes fp32's range; the block's scale, 1, does not.
"""

import pytest
import torch

import sparse_matmul_ffns_amd as nm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BLOCK = 49.0 * 2.0 ** 19


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _ones(rows, K, off=0):
    flat = torch.zeros(off + rows * K, dtype=torch.uint8, device="cuda")
    v = flat[off:].view(rows, K).view(torch.float8_e4m3fn)
    return v.copy_(torch.full((rows, K), 448.0, device="cuda").to(torch.float8_e4m3fn))


def _full(shape, v):
    return torch.full(shape, v, device="cuda")


@pytest.mark.parametrize("ea,eb,want", [(110, -110, 0), (-110, 110, 0), (-126, 100, -26), (60, 40, 100), (120, -1, None)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,off", [(4, 128, 0), (300, 512, 0), (3000, 3328, 0), (140, 256, 1)])
def test_product(M, N, off, block, out, ea, eb, want):
    """The kernels for few rows, for both tile sizes and for unaligned operands."""
    K = 256
    sa, sb = _full((2, M), 2.0 ** ea), _full((2, N) if block == 1 else (N // 128, 2), 2.0 ** eb)
    C = nm.fp8_gemm_nt(_ones(M, K, off), sa, _ones(N, K, off), sb, b_block=block, out_dtype=out)
    v = 2 * BLOCK * 2.0 ** want if want is not None else float("inf")
    assert bool((C.double() == v).all())


@pytest.mark.parametrize("ea,eb", [(110, -110), (-110, 110)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_grouped_products(out, ea, eb):
    off = torch.tensor([0, 256, 256, 640], dtype=torch.int32, device="cuda")
    C = nm.fp8_gemm_nt_grouped(_ones(640, 256), _full((2, 640), 2.0 ** ea), _ones(3 * 256, 256).view(3, 256, 256),
                               _full((3, 2, 2), 2.0 ** eb), off, out_dtype=out)
    assert bool((C.double() == 2 * BLOCK).all())
    C = nm.fp8_gemm_nt_grouped_k(_ones(300, 640), _full((5, 300), 2.0 ** ea), _ones(256, 640), _full((5, 256), 2.0 ** eb),
                                 off, out_dtype=out)
    for e, blocks in enumerate((2, 0, 3)):
        assert bool((C[e].double() == blocks * BLOCK).all())
