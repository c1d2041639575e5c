"""The dense products on operands that the tiled kernels cannot load as they are (rows that do not begin at 16 bytes,
lengths that are no multiple of eight), which are copied into the caller's work memory first; and work memory of any size and
content.  Products of small integers are exact in every order, so every way of computing them gives the same bits.
"""

import pytest
import torch

import sparse_matmul_ffns_amd as nm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _ints(g, R, C, pad=0, off=0):
    """[R, C] with `pad` elements of NaN behind each row and `off` in front of the first."""
    flat = torch.full((off + R * (C + pad) + 16,), float("nan"), device="cuda", dtype=torch.bfloat16)
    t = flat[off:off + R * (C + pad)].view(R, C + pad)[:, :C]
    t.copy_(torch.randint(-3, 4, (R, C), generator=g, device="cuda"))
    return t


def _calls(X, W, D, M, N, K):
    """The three products of a layer: (number of the call, the call with an output and work memory, its value)."""
    dx, dw = D.double() @ W.double(), D.double().t() @ X.double()
    return [(0, lambda y, w: nm.linear_fwd(X, W, out=y, work=w), X.double() @ W.double().t(), (M, N), torch.bfloat16),
            (1, lambda y, w: nm.linear_bwd_x(D, W, out=y, work=w), dx, (M, K), torch.bfloat16),
            (2, lambda y, w: nm.linear_bwd_w(D, X, out=y, work=w), dw, (N, K), torch.float32)]


# M, N, K: whole tiles and ragged ones, long reductions with few tiles (cut into parts besides)
SIZES = [(512, 512, 511), (1000, 1111, 777), (129, 1000, 4001), (4097, 520, 1032), (520, 4097, 264), (513, 1031, 520), (300, 301, 8191),
         (2051, 2053, 331)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("pad,off", [(0, 0), (1, 0), (0, 1), (3, 5), (8, 0)])
def test_copied_operands(M, N, K, pad, off):
    g = torch.Generator(device="cuda").manual_seed(M + N + K + pad)
    X, W, D = _ints(g, M, K, pad, off), _ints(g, N, K, pad, off), _ints(g, M, N, pad, off)
    for which, call, want, shape, dtype in _calls(X, W, D, M, N, K):
        need = nm.nmsparse._linear_work_bytes(which, M, N, K, False)
        for some in ("auto", need, need // 2, 16, None):
            y = torch.full((shape[0], shape[1] + 5), 77.0, device="cuda", dtype=dtype)
            w = some if some in ("auto", None) else torch.full((some + 64,), 255, device="cuda", dtype=torch.uint8)
            call(y[:, :shape[1]], w if some in ("auto", None) else w[:some])
            assert torch.equal(y[:, :shape[1]], want.to(dtype)), (which, some)
            assert bool((y[:, shape[1]:] == 77).all()) and (some in ("auto", None) or bool((w[some:] == 255).all()))


@pytest.mark.parametrize("first", [True, False])
def test_one_operand_of_the_two(first):
    g = torch.Generator(device="cuda").manual_seed(7)
    M, N, K = 600, 712, 1024
    X, W, D = _ints(g, M, K, 0, 3 * first), _ints(g, N, K, 0, 3 * (not first)), _ints(g, M, N, 0, 3 * first)
    for which, call, want, shape, dtype in _calls(X, W, D, M, N, K):
        y = torch.empty(shape, device="cuda", dtype=dtype)
        call(y, "auto")
        assert torch.equal(y, want.to(dtype)), which


def test_epilogues_of_copied_operands():
    g = torch.Generator(device="cuda").manual_seed(8)
    M, N, K = 700, 1001, 1203
    X, W, R, D = _ints(g, M, K), _ints(g, N, K), _ints(g, M, N, 3, 1), _ints(g, M, N)
    b = _ints(g, 1, N)[0]
    z = X.double() @ W.double().t() + b.double()
    P = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    Y, _ = nm.linear_fwd(X, W, bias=b, act="relu", residual=R, pre=P)
    assert torch.equal(P, z.bfloat16()) and torch.equal(Y, (z.clamp(min=0) + R.double()).bfloat16())
    Q = _ints(g, M, K, 1)
    dx = D.double() @ W.double()
    assert torch.equal(nm.linear_bwd_x(D, W, pre=Q, act="relu"), torch.where(Q > 0, dx, torch.zeros_like(dx)).bfloat16())
    dW = torch.ones(N, K, device="cuda")
    nm.linear_bwd_w(D, X, out=dW, accumulate=True)
    assert torch.equal(dW, (1 + D.double().t() @ X.double()).float())


def test_values_that_are_not_finite_stay_in_their_rows():
    """Zeros behind a copy's rows meet values of the other operand: none of its rows may become NaN by that."""
    g = torch.Generator(device="cuda").manual_seed(9)
    M, N, K = 400, 530, 1029
    X, W = _ints(g, M, K), _ints(g, N, K)
    want = X.double() @ W.double().t()
    X[5, K - 1] = float("inf")
    X[9, 0] = float("nan")
    Y = nm.linear_fwd(X, W)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[5] = keep[9] = False
    assert torch.equal(Y[keep], want[keep].bfloat16()) and bool(Y[9].isnan().all()) and not bool(Y[5].isfinite().any())


@pytest.mark.parametrize("M,N,K", [(300, 264, 512), (70, 33, 41), (5, 8, 16)])
def test_what_relu_masks_goes_no_further(M, N, K):
    """An infinite or undefined gradient where ReLU let nothing through: 0, in the products' epilogues too."""
    g = torch.Generator(device="cuda").manual_seed(11)
    D, W, P, dY = _ints(g, M, N), _ints(g, N, K), _ints(g, M, K), _ints(g, M, K)
    bad = dY.clone()
    bad[P <= 0] = float("inf")
    bad[3, :][P[3] <= 0] = float("nan")
    (dZ, db), (dz, d) = nm.linear_bwd_act(bad, P, act="relu"), nm.linear_bwd_act(dY, P, act="relu")
    assert torch.equal(dZ, dz) and torch.equal(db, d) and bool(dz.isfinite().all())
    want = nm.linear_bwd_x(D, W, pre=P, act="relu")
    D[3, 0] = float("inf")                                # row 3 of the product is not finite
    W[0] = W[0].abs() + 1
    P[3] = -1
    want[3] = 0
    got = nm.linear_bwd_x(D, W, pre=P, act="relu")
    assert torch.equal(got[3], want[3])


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32])
@pytest.mark.parametrize("K", [1, 7, 8, 31, 33, 777, 2047])
def test_few_rows_of_any_alignment(M, K):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    for N, pad, off in ((1, 0, 0), (37, 0, 0), (530, 3, 1)):
        X, W = _ints(g, M, K, pad, off), _ints(g, N, K, pad, off)
        assert torch.equal(nm.linear_fwd(X, W), (X.double() @ W.double().t()).bfloat16()), N


def test_in_a_graph_with_its_own_work():
    g = torch.Generator(device="cuda").manual_seed(10)
    M, N, K = 300, 301, 8191
    X, W, D = _ints(g, M, K), _ints(g, N, K), _ints(g, M, N)
    calls = _calls(X, W, D, M, N, K)
    outs = [torch.zeros(shape, device="cuda", dtype=dtype) for _, _, _, shape, dtype in calls]
    works = [torch.full((max(nm.nmsparse._linear_work_bytes(c[0], M, N, K, False), 1),), 255, device="cuda", dtype=torch.uint8) for c in calls]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        for c, y, w in zip(calls, outs, works):
            c[1](y, w)
    for seed in range(3):
        g.manual_seed(seed)
        for t in (X, W, D):
            t.copy_(torch.randint(-3, 4, t.shape, generator=g, device="cuda"))
        for y, w in zip(outs, works):
            y.zero_()
            w.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for c, y in zip(_calls(X, W, D, M, N, K), outs):
            assert torch.equal(y, c[2].to(y.dtype)), (seed, c[0])
