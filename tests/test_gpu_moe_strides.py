"""Operands and outputs with other row strides and alignments, in every mixture-of-experts call (GPU): the
result has to be that of contiguous operands bit for bit, and nothing outside the output's rows may change.
(The products' unaligned operands take another kernel, which sums in another order: there small integers
and powers of two make every sum exact.)
"""

import numpy as np
import pytest
import torch

import sparse_matmul_ffns_amd as nm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
CANARY = 0x5A


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


class View:
    """A [rows, cols] view at `off` elements into a buffer of canary bytes, `pad` elements behind each row."""

    def __init__(self, rows, cols, dtype, pad, off, values=None):
        size = torch.empty(0, dtype=dtype).element_size()
        self.bytes = torch.full(((off + rows * (cols + pad)) * size,), CANARY, dtype=torch.uint8, device="cuda")
        wide = self.bytes.view(dtype)[off:].view(rows, cols + pad)
        self.t = wide[:, :cols]
        if values is not None:
            self.t.copy_(values)

    def untouched(self):
        """True if the bytes outside the view are the canary's still."""
        size, (rows, cols), ld = self.t.element_size(), self.t.shape, self.t.stride(0)
        outside = torch.ones_like(self.bytes, dtype=torch.bool)
        first = outside.numel() - rows * ld * size
        outside[first:].view(rows, ld * size)[:, :cols * size] = False
        return bool((self.bytes[outside] == CANARY).all())


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _same(a, b):
    return torch.equal(_bits(a), _bits(b))


LAYOUTS = [(0, 0), (1, 0), (0, 1), (3, 1), (8, 8), (16, 0), (5, 3)]      # pad, off


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(37, 64, 8), (19, 60, 6), (9, 256, 20), (5, 300, 3)])
def test_route(T, E, k, dtype):
    logits, dw = _rand(1, T, E).to(dtype), _rand(2, T, k)
    for score, renorm, b in (("softmax", False, None), ("sigmoid", True, _rand(3, E) * 0.01)):
        ids, w = nm.moe_route(logits, k, score=score, renorm=renorm, bias=b)
        dl = nm.moe_route_bwd(logits, ids, w, dw, score=score, renorm=renorm)
        for pad, off in LAYOUTS:
            l = View(T, E, dtype, pad, off, logits)
            shifted = None if b is None else torch.cat([b[:off], b])[off:]      # off a 16-byte boundary
            i2, w2 = nm.moe_route(l.t, k, score=score, renorm=renorm, bias=shifted)
            assert torch.equal(i2, ids) and _same(w2, w)
            out = View(T, E, dtype, pad, off)
            nm.moe_route_bwd(l.t, ids, w, dw, score=score, renorm=renorm, dlogits=out.t)
            assert _same(out.t, dl) and out.untouched()


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,K", [(5, 8), (130, 264), (33, 201)])
def test_quantize(R, K, dtype, fmt):
    X, G = _rand(1, R, K).to(dtype), _rand(2, R, K).to(dtype)
    for t, call in ((False, nm.fp8_quantize), (True, nm.fp8_quantize_t)):
        q, s = call(X, fmt, gate=G)
        for pad, off in LAYOUTS:
            x, g = View(R, K, dtype, pad, off, X), View(R, K, dtype, (pad + 3) % 9, off, G)
            Q, S = View(*q.shape, fmt, pad, off), View(*s.shape, torch.float32, pad, off)
            call(x.t, fmt, gate=g.t, Q=Q.t, S=S.t)
            assert _same(Q.t, q) and _same(S.t, s), (t, pad, off)
            assert Q.untouched() and S.untouched()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(130, 264), (3, 7)])
def test_quantize_weight(N, K, dtype):
    E = 3
    W = _rand(1, E * N, K).to(dtype)
    want = nm.fp8_quantize_weight(W.view(E, N, K), transposed=True)
    for pad, off in LAYOUTS:
        w = View(E * N, K, dtype, pad, off, W).t
        got = nm.fp8_quantize_weight(w.unflatten(0, (E, N)), transposed=True)
        assert all(_same(a, b) for a, b in zip(got, want)), (pad, off)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(3, 200, 264), (130, 264, 130), (700, 136, 384)])
def test_products(M, N, K, out):
    f8, Kb = torch.float8_e4m3fn, -(-K // 128)
    ints = lambda seed, *s: _rand(seed, *s).mul(1.5).round().clamp(-3, 3)
    power = lambda seed, *s: 2.0 ** _rand(seed, *s).round().clamp(-2, 2)
    A, B, sa = ints(1, M, K).to(f8), ints(2, 3 * N, K).to(f8), power(3, Kb, M)
    sbr, sbb = power(4, Kb, N), power(5, 3, -(-N // 128), Kb)
    off = torch.tensor([0, M // 3, M // 3, M - 1], dtype=torch.int32, device="cuda")
    want = [nm.fp8_gemm_nt(A, sa, B[:N], sbb[0], out_dtype=out), nm.fp8_gemm_nt(A, sa, B[:N], sbr, b_block=1, out_dtype=out),
            nm.fp8_gemm_nt_grouped(A, sa, B.view(3, N, K), sbb, off, out_dtype=out)]
    for pad, o in LAYOUTS:
        a, b, s = View(M, K, f8, pad, o, A).t, View(3 * N, K, f8, (pad + 8) % 17, o, B).t, View(Kb, M, torch.float32, pad, o, sa).t
        r, blk = View(Kb, N, torch.float32, pad, o, sbr).t, View(*sbb[0].shape, torch.float32, pad, o, sbb[0]).t
        C = [View(M, N, out, pad, o) for _ in range(3)]
        nm.fp8_gemm_nt(a, s, b[:N], blk, out=C[0].t)
        nm.fp8_gemm_nt(a, s, b[:N], r, b_block=1, out=C[1].t)
        nm.fp8_gemm_nt_grouped(a, s, b.unflatten(0, (3, N)), sbb, off, out=C[2].t)
        for c, w in zip(C, want):
            assert torch.equal(c.t, w), (pad, o)       # a sum of zeros may be -0
            assert c.untouched()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products_over_groups_of_the_reduction(out):
    f8, M, N, R = torch.float8_e4m3fn, 130, 72, 640
    ints = lambda seed, *s: _rand(seed, *s).mul(1.5).round().clamp(-3, 3)
    power = lambda seed, *s: 2.0 ** _rand(seed, *s).round().clamp(-2, 2)
    A, B, sa, sb = ints(1, M, R).to(f8), ints(2, N, R).to(f8), power(3, R // 128, M), power(4, R // 128, N)
    off = torch.tensor([0, 256, 256, 512], dtype=torch.int32, device="cuda")
    want = nm.fp8_gemm_nt_grouped_k(A, sa, B, sb, off, out_dtype=out)
    for pad, o in LAYOUTS:
        C = nm.fp8_gemm_nt_grouped_k(View(M, R, f8, pad, o, A).t, View(*sa.shape, torch.float32, pad, o, sa).t,
                                     View(N, R, f8, (pad + 8) % 17, o, B).t, View(*sb.shape, torch.float32, pad, o, sb).t, off,
                                     out_dtype=out)
        assert torch.equal(C, want), (pad, o)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,D", [(7, 3, 16), (40, 8, 513), (3, 2, 2500)])
def test_combine(T, k, D, dtype):
    ids = torch.from_numpy(np.random.default_rng(1).integers(-1, 6, size=(T, k)).astype(np.int32)).cuda()
    _, _, src, pos = nm.moe_plan(ids, 6, 16)
    rows = src.numel()
    O, dY, w = _rand(1, rows, D).to(dtype), _rand(2, T, D).to(dtype), _rand(3, T, k)
    want = nm.moe_combine(O, pos, w)
    dO, dw = nm.moe_combine_bwd(dY, O, src, pos, w)
    for pad, off in LAYOUTS:
        o, dy = View(rows, D, dtype, pad, off, O).t, View(T, D, dtype, (pad + 3) % 9, off, dY).t
        Y, G = View(T, D, dtype, pad, off), View(rows, D, dtype, pad, off)
        nm.moe_combine(o, pos, w, out=Y.t)
        assert _same(Y.t, want) and Y.untouched()
        _, gw = nm.moe_combine_bwd(dy, o, src, pos, w, dO=G.t)
        assert _same(G.t, dO) and G.untouched()
        # dweights: the columns are dealt to the lanes alike, so the sums are the same
        assert _same(gw, dw)
