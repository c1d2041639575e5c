"""The dense product of one row (a token) along its whole reduction (GPU): every number of waves, trips of the loop and tails.

Tolerances (U = 2^-24): a product of bf16 values is exact in fp32 and each of the K additions rounds once, (K + 4) U of sum |x| |w|; an
activation has a slope below 1.2."""

import numpy as np
import pytest
import torch

import sparse_matmul_ffns_amd as nm
from oracle import dense_oracle as O
from tests.gpu_util import require_gpu
from tests.test_gpu_dense import TD, U, buffer, close, dev, half, host

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _ints(rng, *shape):
    return rng.integers(-3, 4, size=shape).astype(np.float64)


# one wave and two chunks up to eight waves, 512 threads from 7169 on, a second trip behind 8192, trips whose second chunk is missing or
# odd; three rows of B behind the last four, and none
@pytest.mark.parametrize("K", [1, 7, 511, 513, 1025, 2049, 4096, 7168, 7169, 8191, 8192, 8193, 8200, 12288, 12289, 16384, 16391, 24577])
@pytest.mark.parametrize("N,pad,off", [(96, 0, 0), (67, 5, 3), (1, 8, 1)])
def test_one_row(K, N, pad, off):
    """Small integers: sums up to 9 K stay below 2^24, so every order of adding gives the same bits."""
    rng = np.random.default_rng(K + N)
    X, x = dev(_ints(rng, 1, K), "bf16", pad, off)
    W, w = dev(_ints(rng, N, K), "bf16", pad, off)
    z = x @ w.T
    Y, intact = buffer(1, N, torch.float32, pad, off)
    assert nm.linear_fwd(X, W, out=Y) is Y and intact()
    assert np.array_equal(host(Y), z)
    B, b = dev(_ints(rng, N), "f32", 0, off)
    R, r = dev(_ints(rng, 1, N), "bf16", pad, off)
    for out in ("bf16", "f32"):
        Y, intact = buffer(1, N, TD[out], pad, off)
        P, intact_p = buffer(1, N, torch.bfloat16, pad, off)
        nm.linear_fwd(X, W, bias=B, act="relu", residual=R, out=Y, pre=P)
        assert intact() and intact_p()
        assert np.array_equal(host(P), torch.from_numpy(z + b).bfloat16().double().numpy())
        assert np.array_equal(host(Y), torch.from_numpy(np.maximum(z + b, 0) + r).to(TD[out]).double().numpy())


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu"])
@pytest.mark.parametrize("N,K", [(130, 8193), (64, 16384), (33, 7169)])
def test_one_row_of_real_values(N, K, act):
    rng = np.random.default_rng(N + K)
    X, x = dev(rng.normal(size=(1, K)))
    W, w = dev(rng.normal(size=(N, K)) * 1.5 / np.sqrt(K))
    B, b = dev(rng.normal(size=N))
    y, z = O.linear(x, w, b, act)
    ez = (K + 4) * U * (np.abs(x) @ np.abs(w).T) + 2 * U * np.abs(z)
    got, pre = nm.linear_fwd(X, W, bias=B, act=act, out_dtype=torch.float32, return_pre=True)
    close(pre, z, ez + half(z, "bf16") * 1.01, "pre")
    close(got, y, 1.2 * ez + O.act_error(z, act) + 2 * U * np.abs(y), "y")
    assert torch.equal(got, nm.linear_fwd(X, W, bias=B, act=act, out_dtype=torch.float32))
