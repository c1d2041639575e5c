"""A product whose operands' copies take more work-items than a launch holds (GPU): 2^30 rows of 17 and of 9 columns, 141 GB."""

import pytest
import torch

import sparse_matmul_ffns_amd as nm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def test_weight_gradient_of_2_30_rows():
    require_gpu()
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 200 GB of GPU memory")
    M, N, K = 1 << 30, 17, 9
    D = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    X = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    # a launch's copies end behind 2^31 groups: in row 2^31 / 3 of D, and 2^32 in X's row 2^29
    at = torch.tensor([0, 1, (1 << 31) // 3 - 1, (1 << 31) // 3, (1 << 31) // 3 + 1, (1 << 29) - 1, 1 << 29, (1 << 29) + 1, M // 16, M - 2, M - 1],
                      device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    D[at] = torch.randint(-3, 4, (len(at), N), generator=g, device="cuda").bfloat16()
    X[at] = torch.randint(-3, 4, (len(at), K), generator=g, device="cuda").bfloat16()
    want = D[at].double().t() @ X[at].double()
    torch.cuda.synchronize()
    got = nm.linear_bwd_w(D, X)
    torch.cuda.synchronize()
    assert torch.equal(got.double(), want)
    del D, X, got
    torch.cuda.empty_cache()
