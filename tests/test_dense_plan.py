"""Calls whose copies of unaligned operands take more work-items than a launch (C ABI; CPU: a call that can be launched ends with HIP's
'no device', one whose launch does not fit with 'invalid configuration')."""

import ctypes
import os

import pytest

from sparse_matmul_ffns_amd import nmsparse as nm

pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="runs only where no GPU is visible: the addresses are made up")
A, B, C, W = ((1 << 45) * i for i in range(1, 5))


@pytest.fixture(scope="module")
def L():
    return nm.lib()


def _no_device(L, status):
    return status == nm.NM_ERR_HIP and b"invalid configuration" not in L.nm_last_hip_error()


# groups of eight of a row: 256 in 2041 columns, two in 9; the copies take 2^32 work-items from 2^24 and 2^30 rows on
@pytest.mark.parametrize("M", [(1 << 24) - 2000, (1 << 24) - 1, 1 << 24, (1 << 24) + 5, 1 << 25, (1 << 31) - 1])
@pytest.mark.parametrize("with_work", [True, False])
def test_rows_of_2041(L, M, with_work):
    N, K = 1000, 2041
    need = ctypes.c_int64()
    for call in (0, 1):
        sizes = (M, N, K) if call == 0 else (M, K, N)
        assert L.linear_work_bytes(call, *sizes, 0, ctypes.byref(need)) == nm.NM_OK
        assert need.value >= 2 * min(M, 1 << 24) * 2048          # the copy is planned
        work, room = (W, need.value) if with_work else (None, 0)
        if call == 0:
            st = L.linear_fwd(1, A, K, B, K, 1, None, 0, None, 0, M, N, K, 1, C, N, None, 0, work, room, None)
        else:
            st = L.linear_bwd_x(1, A, K, B, N, None, 0, 0, M, K, N, 1, C, N, work, room, None)
        assert _no_device(L, st), (call, L.nm_last_hip_error())


@pytest.mark.parametrize("M", [(1 << 30) - 200, 1 << 30, (1 << 30) + 1, (1 << 31) - 1])
@pytest.mark.parametrize("N", [9, 17])
def test_reductions_over_2_30_rows(L, M, N):
    K, need = 9, ctypes.c_int64()
    assert L.linear_work_bytes(2, M, N, K, 0, ctypes.byref(need)) == nm.NM_OK
    st = L.linear_bwd_w(1, A, N, B, K, M, N, K, 0, 0, C, K, W if need.value else None, need.value, None)
    assert _no_device(L, st), L.nm_last_hip_error()
