"""The mixture-of-experts FFN in 8 bits against its fp64 oracle (GPU).

Tolerances, from the arithmetic: routing weights are quotients of fp32 exponentials of rounded
differences |l - max| < 64 (relative error below 64 * 2^-24 * 2 in each) and sums of at most 1024 terms
in at most 26 rounded steps: 1e-5 relative.  The gradient's terms are products of those: 2e-5 of the sum
of their magnitudes, plus half a unit in the last place of a bf16 result (2^-8 relative).  An 8-bit
product with a bf16 result adds 128 terms in the matrix instruction, each aligned to the block's largest,
which keeps at least 12 bits below it per term, then scales and adds fp32 blocks: |C - C*| <= 2^-12
sum_kb (|A| |B|)_kb plus half a unit of the result.  With an fp32 result the 128 products and their sums
are fp32: 128 * 2^-24 + (blocks + 2) * 2^-24 of sum_kb (|A| |B|)_kb.  Products of small integers are exact.  Quantisation, orders and ids
are exact.  The combine adds k <= 64 fp32 products: 64 * 2^-24 of the sum of magnitudes.
"""

import numpy as np
import pytest
import torch

import sparse_matmul_ffns_amd as nm
from oracle import moe_oracle as MO
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
T8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def dev(a, dtype="f32", pad=0):
    """float64 array -> (device tensor, the float64 values it holds); `pad` extra columns (NaN) behind each row."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TD[dtype])
    if pad:
        wide = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=t.dtype)
        wide[:, :a.shape[1]] = t
        return wide.cuda()[:, :a.shape[1]], t.double().numpy()
    return t.cuda(), t.double().numpy()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def host(t):
    return t.detach().cpu().double().numpy()


def bytes_of(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def fp8_dev(q, fmt, pad=0, off=0):
    """uint8 array -> device 8-bit tensor; `pad` bytes of NaN behind each row, `off` bytes off alignment."""
    r, c = q.shape
    flat = torch.full((off + r * (c + pad),), 0x7F, dtype=torch.uint8, device="cuda")
    v = flat[off:].view(r, c + pad)
    v[:, :c] = torch.from_numpy(q).cuda()
    return v[:, :c].view(T8[fmt]) if pad == 0 else v.view(T8[fmt])[:, :c]


def half_ulp(x, dtype):
    return np.abs(x) * 2.0 ** -8 if dtype == "bf16" else 0.0


# ---- routing ------------------------------------------------------------------------------------
def _logits(rng, T, E, kind):
    l = rng.normal(size=(T, E)) * 2
    if kind == "ties":
        l = np.round(l)
    if kind == "masked":
        l[rng.random((T, E)) < 0.5] = -np.inf
        l[0] = -np.inf                                    # a row with nothing
        if T > 1:
            l[1] = -np.inf
            l[1, E // 2] = 3.0                            # a row with one
        if T > 2:
            l[2] = -3.3895313892515355e38                 # the lowest bf16
        if T > 3:
            l[3, ::2] = -3.3895313892515355e38
        if T > 4:
            l[4, 0], l[4, E - 1] = np.nan, np.inf
    return l


ROUTE = [
    # T, E, k, groups, topk_groups, group_top
    (1, 1, 1, 1, 1, 2), (3, 2, 2, 1, 1, 2), (5, 8, 2, 1, 1, 2), (1, 64, 8, 1, 1, 2), (17, 60, 4, 1, 1, 2),
    (33, 65, 7, 1, 1, 2), (9, 160, 6, 8, 3, 1), (67, 256, 8, 8, 4, 2), (21, 256, 16, 4, 1, 2), (6, 256, 20, 1, 1, 2),
    (13, 300, 64, 3, 2, 2), (5, 1024, 10, 64, 4, 2), (7, 64, 3, 64, 5, 2),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked"])
@pytest.mark.parametrize("case", ROUTE)
def test_route(case, kind, score):
    T, E, k, groups, tg, gt = case
    rng = np.random.default_rng(1000 * T + E + k + len(kind) + len(score))
    for dtype, renorm, bias, pad in (("bf16", True, False, 0), ("f32", False, False, 3), ("f32", True, True, 0),
                                     ("bf16", False, True, 5)):
        dl, l = dev(_logits(rng, T, E, kind), dtype, pad)
        b = db = None
        if bias:
            b = np.round(rng.normal(size=E) * 20) * 2.0 ** -10
            db, b = dev(b)
        ids, w, S = MO.route(l, k, score, b, groups, tg, gt, renorm, 1.5)
        # where 64-bit scores differ by less than 2e-6 of the largest without being equal in their inputs,
        # fp32 may order them otherwise: there the chosen experts' scores are compared, not their ids
        # (and nothing where the groups' scores are that close)
        near = np.array([_near(l[t], S[t], b, groups, gt) for t in range(T)])
        keep = near == 0
        gi, gw = nm.moe_route(dl, k, score=score, bias=db, groups=groups, topk_groups=tg, group_top=gt, renorm=renorm,
                              scale=1.5)
        gi, gw = gi.cpu().numpy(), host(gw)
        assert np.array_equal(gi[keep], ids[keep]), (dtype, renorm, bias)
        for t in np.nonzero(near == 1)[0]:
            c = S[t] if b is None else S[t] + b
            assert ((gi[t] < 0) == (ids[t] < 0)).all() and len(set(gi[t])) == len(set(ids[t]))
            live = gi[t] >= 0
            assert (np.abs(c[gi[t][live]] - c[ids[t][live]]) <= 2e-6 * np.abs(c).max()).all()
        assert (np.abs(gw - w)[keep] <= 1e-5 * np.abs(w)[keep] + 1e-37).all(), (dtype, renorm, bias)
        assert (gw[gi < 0] == 0).all()


def _near(l, s, b, groups, gt):
    """1: two scores, 2: two groups' scores that fp32 may order otherwise."""
    ok = ~np.isnan(l) & (l > -np.inf)
    c = (s if b is None else s + b)[ok]
    if c.size < 2:
        return 0
    key = list(zip(np.minimum(l[ok], np.finfo(np.float32).max), b[ok] if b is not None else np.zeros(c.size)))
    o = np.argsort(-c, kind="stable")
    lim = 2e-6 * np.abs(c).max()
    out = 0
    if b is not None and any(c[o[i]] - c[o[i + 1]] < lim and key[o[i]] != key[o[i + 1]] for i in range(c.size - 1)):
        out = 1
    if groups > 1:
        n = l.size // groups
        full = np.where(ok, s if b is None else s + b, -np.inf)
        sc = []
        for g in range(groups):
            top = np.sort(full[g * n:(g + 1) * n])[::-1][:gt]
            top = top[top > -np.inf]
            sc.append((top.sum() if top.size else -np.inf, tuple(np.sort(l[g * n:(g + 1) * n])[::-1][:gt])))
        sc.sort(key=lambda x: -x[0])
        if any(sc[i][0] - sc[i + 1][0] < 2 * lim and (sc[i][1] != sc[i + 1][1] or b is not None)
               for i in range(groups - 1) if sc[i + 1][0] > -np.inf):
            return 2
    return out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("case", [(1, 64, 8), (3, 1, 1), (19, 60, 5), (50, 256, 8), (6, 256, 30), (4, 1000, 33)])
def test_route_bwd(case, renorm, score):
    T, E, k = case
    rng = np.random.default_rng(T * E + k)
    for dtype, pad in (("f32", 0), ("bf16", 0), ("f32", 1)):
        l = _logits(rng, T, E, "normal")
        if T > 4:
            l[0] = -np.inf
            l[1, 1:] = -np.inf
            l[2, ::3] = -np.inf
        dl, l = dev(l, dtype, pad)
        ids, w, _ = MO.route(l, k, score, renorm=renorm, scale=2.5)
        gw, w = dev(w)
        dw_, dw = dev(rng.normal(size=(T, k)))
        want = MO.route_bwd(l, ids, w, dw, score, renorm, 2.5)
        got = host(nm.moe_route_bwd(dl, i32(ids), gw, dw_, score=score, renorm=renorm, scale=2.5))
        mag = (np.abs(w * dw).sum(1, keepdims=True) / 2.5 + np.abs(dw).max(1, keepdims=True)) * 2.5
        s = np.zeros((T, E))
        for t in range(T):
            s[t, ids[t][ids[t] >= 0]] = w[t][ids[t] >= 0] / 2.5
        # the chosen entries' own weights bound the terms; plain softmax spreads the sum over every s_e
        scale = s * mag if (renorm or score == "sigmoid") else mag
        assert (np.abs(got - want) <= 2e-5 * scale + half_ulp(want, dtype) + 1e-30).all()
        if renorm or score == "sigmoid":
            assert (got[s == 0] == 0).all()


def test_route_bwd_ignores_ids_outside():
    l, _ = dev(np.zeros((2, 8)))
    ids = i32([[-1, 9], [3, -5]])
    w, _ = dev(np.full((2, 2), 0.5))
    d = host(nm.moe_route_bwd(l, ids, w, torch.ones(2, 2, device="cuda"), renorm=False))
    assert (d[0] == 0).all() and d[1, 3] > 0


# ---- plan ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (5, 3, 7), (513, 8, 60), (4096, 1, 256), (700, 6, 1024),
                                   (1025, 8, 64), (20001, 7, 160), (131072, 10, 8)])
@pytest.mark.parametrize("align", [1, 16, 128, 256])
def test_plan(T, k, E, align):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    if T > 4:
        ids[rng.random((T, k)) < 0.1] = -1
        ids[T // 2] = E + 3
        ids[ids == E // 2] = 0                                 # an expert with nothing
    rows = nm.moe_plan_rows(T * k, E, align)
    want = MO.plan(ids, E, align, rows)
    got = nm.moe_plan(i32(ids), E, align)
    for g, w, name in zip(got, want, ("offsets", "counts", "src", "pos")):
        assert np.array_equal(g.cpu().numpy(), w), name
    # more rows than needed
    src = torch.full((rows + 777,), 5, dtype=torch.int32, device="cuda")
    got = nm.moe_plan(i32(ids), E, align, src=src)
    assert np.array_equal(got[2].cpu().numpy(), np.concatenate([want[2], np.full(777, -1, np.int32)]))


# ---- quantisation -------------------------------------------------------------------------------
def _wild(rng, R, K, dtype):
    x = rng.normal(size=(R, K)) * np.exp(rng.normal(size=(R, 1)) * 4) * np.exp(rng.normal(size=(1, K)))
    x[rng.random((R, K)) < 0.1] = 0.0
    if R > 3 and K > 3:
        x[0] = 0.0
        x[1, 0], x[1, 1], x[2, 2] = np.nan, np.inf, -np.inf
        x[3] = 1e-42 if dtype == "f32" else 1e-39              # subnormal
        x[-1] = 448.0 * 2.0 ** 5
        x[-1, -1] = 449.0 * 2.0 ** 5 if dtype == "f32" else 452.0 * 2.0 ** 5
    return x


QUANT = [(1, 1), (4, 128), (7, 130), (33, 200), (128, 256), (129, 264), (40, 1000), (260, 72)]


def _check_bytes(got, want, fmt):
    v = MO.decode8(fmt)
    a, b = v[got], v[want]
    assert np.array_equal(a, b, equal_nan=True)
    assert np.array_equal(np.signbit(a)[~np.isnan(a)], np.signbit(b)[~np.isnan(b)])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("R,K", QUANT)
def test_quantize(R, K, fmt):
    rng = np.random.default_rng(R * K)
    for dtype, pad, gather, gated in (("bf16", 0, False, False), ("f32", 0, True, False), ("bf16", 8, True, True),
                                      ("bf16", 3, False, True), ("f32", 1, False, False)):
        dx, x = dev(_wild(rng, R, K, dtype), dtype, pad)
        src = dsrc = dg = g = None
        n, div = R, 1
        if gather:
            n, div = 2 * R + 5, 3
            src = rng.integers(-1, R * div + 4, size=n).astype(np.int32)
            dsrc = i32(src)
        if gated:
            dg, g = (dx, x) if not gather else dev(rng.normal(size=(n, K)), dtype, pad)
        y = MO.rows_of(x, src, div, g)
        for t in (False, True):
            want = MO.quantize(np.ascontiguousarray(y.T) if t else y, fmt)
            call = nm.fp8_quantize_t if t else nm.fp8_quantize
            q, s = call(dx, T8[fmt], src=dsrc, div=div, gate=dg)
            assert np.array_equal(host(s), want[1]), (dtype, t)
            _check_bytes(bytes_of(q), want[0], fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (1, 128, 128), (3, 200, 130), (2, 72, 300)])
def test_quantize_weight(E, N, K, fmt):
    rng = np.random.default_rng(N * K)
    for dtype in ("bf16", "f32"):
        dw, w = dev(np.concatenate([_wild(rng, N, K, dtype) for _ in range(E)]), dtype)
        q, s, qt, st = nm.fp8_quantize_weight(dw.view(E, N, K), T8[fmt], transposed=True)
        for e in range(E):
            wq, ws = MO.quantize_weight(w.reshape(E, N, K)[e], fmt)
            assert np.array_equal(host(s[e]), ws) and np.array_equal(host(st[e]), ws.T)
            _check_bytes(bytes_of(q[e]), wq, fmt)
            b = bytes_of(qt[e])
            _check_bytes(b[:, :N], np.ascontiguousarray(wq[:, :K].T), fmt)
            assert (b[:, N:] == 0).all()
    q2, s2 = nm.fp8_quantize_weight(dw.view(E, N, K)[0], T8[fmt])
    assert torch.equal(q2.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s2, s[0])


# ---- products -----------------------------------------------------------------------------------
def _bytes(rng, R, K, fmt, kind):
    if kind == "ints":
        return MO.encode8(rng.integers(-3, 4, size=(R, K)).astype(float), fmt)
    x = rng.normal(size=(R, K))
    return MO.encode8(x / np.abs(x).max() * MO.MAX8[fmt] * (1.0 if kind == "normal" else 2.0 ** -8), fmt)


def _scale_of(rng, shape, kind):
    return (2.0 ** rng.integers(-3, 3, size=shape)) if kind == "ints" else rng.uniform(0.5, 2.0, size=shape).astype(np.float32)


def _ref(A, B, lo=0, hi=None):
    """C* and sum_kb (|A| |B|): in fp64 from the operands' values."""
    return A @ B.T, np.abs(A) @ np.abs(B).T


def _check_product(got, ref, mag, dtype, kind, what, blocks=64):
    if kind == "ints" and dtype == "f32":
        assert np.array_equal(got, ref), what
    else:
        tol = mag * (2.0 ** -12 if dtype == "bf16" else (130 + blocks) * 2.0 ** -24) + half_ulp(ref, dtype) + 1e-30
        assert (np.abs(got - ref) <= tol).all(), (what, (np.abs(got - ref) / tol).max())


GEMM = [(1, 1, 1), (1, 128, 128), (1, 200, 2048), (2, 64, 256), (3, 1000, 130), (16, 129, 512), (17, 257, 384),
        (33, 136, 640), (64, 512, 1024), (65, 300, 200), (127, 128, 4096), (129, 260, 144), (256, 256, 128),
        (300, 520, 1040), (513, 384, 272), (1100, 1030, 400)]


@pytest.mark.parametrize("M,N,K", GEMM)
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_gemm(M, N, K, fa, fb):
    rng = np.random.default_rng(M + N + K)
    Kb, Nb = -(-K // 128), -(-N // 128)
    for kind, out, block, pad, off in (("ints", "f32", 128, 0, 0), ("normal", "bf16", 128, -K % 16, 0),
                                       ("normal", "f32", 1, -K % 128 + 128, 0), ("ints", "f32", 1, 0, 1),
                                       ("ints", "f32", 1, -K % 16 + 16, 0)):
        qa, qb = _bytes(rng, M, K, fa, kind), _bytes(rng, N, K, fb, kind)
        sa = _scale_of(rng, (Kb, M), kind)
        sb = _scale_of(rng, (Kb, N) if block == 1 else (Nb, Kb), kind)
        a = MO.values_rows(qa, sa, fa)
        b = MO.values_rows(qb, sb, fb) if block == 1 else MO.values_blocks(qb, sb, fb)
        C = nm.fp8_gemm_nt(fp8_dev(qa, fa, pad, off), dev(sa)[0], fp8_dev(qb, fb, pad, off), dev(sb)[0], b_block=block,
                           out_dtype=TD[out])
        _check_product(host(C), *_ref(a, b), out, kind, (kind, out, block, pad, off))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
def test_gemm_many_stages_and_tiles(fa, block, out):
    """Hundreds of workgroups over 64 stages whose scales differ from stage to stage: a scale or an operand
    read after its buffer was refilled changes integers that are compared exactly (bf16: powers of two
    small enough that the sums are within 2^-8)."""
    rng = np.random.default_rng(9)
    M, N, K = 2048, 2304, 8192
    qa, qb = _bytes(rng, M, K, fa, "ints"), _bytes(rng, N, K, "e4m3", "ints")
    sa = _scale_of(rng, (K // 128, M), "ints")
    sb = _scale_of(rng, (K // 128, N) if block == 1 else (N // 128, K // 128), "ints")
    a, b = MO.values_rows(qa, sa, fa), MO.values_rows(qb, sb, "e4m3") if block == 1 else MO.values_blocks(qb, sb, "e4m3")
    ref = (torch.from_numpy(a).cuda() @ torch.from_numpy(b).cuda().t()).cpu().numpy()
    args = fp8_dev(qa, fa), dev(sa)[0], fp8_dev(qb, "e4m3"), dev(sb)[0]
    for _ in range(3):
        C = host(nm.fp8_gemm_nt(*args, b_block=block, out_dtype=TD[out]))
        if out == "f32":
            assert np.array_equal(C, ref)
        else:
            assert (np.abs(C - ref) <= np.abs(ref) * 2.0 ** -8).all()


def test_gemm_strided_output_and_scales():
    rng = np.random.default_rng(4)
    M, N, K = 70, 301, 256
    qa, qb = _bytes(rng, M, K, "e4m3", "ints"), _bytes(rng, N, K, "e4m3", "ints")
    sa, sb = _scale_of(rng, (2, M), "ints"), _scale_of(rng, (3, 2), "ints")
    for cdt in ("f32", "bf16"):
        for width, shift in ((N + 3, 0), (N + 3, 1), (N + 8, 0)):
            buf = torch.full((M, width + shift), 7.0, dtype=TD[cdt], device="cuda")
            out = buf[:, shift:shift + N]
            nm.fp8_gemm_nt(fp8_dev(qa, "e4m3"), dev(sa, pad=5)[0], fp8_dev(qb, "e4m3"), dev(sb, pad=2)[0], out=out)
            ref, mag = _ref(MO.values_rows(qa, sa, "e4m3"), MO.values_blocks(qb, sb, "e4m3"))
            _check_product(host(out), ref, mag, cdt, "ints", (cdt, width, shift))
            rest = torch.cat([buf[:, :shift], buf[:, shift + N:]], 1)
            assert bool((rest == 7.0).all())


def _grouped_offsets(rng, E, rows, align, empties=True):
    cut = np.sort(rng.integers(0, rows // align + 1, size=E + 1)) * align
    if empties and E > 2:
        cut[1] = cut[0]
        cut[-1] = cut[-2]
    return cut.astype(np.int32)


@pytest.mark.parametrize("E,rows,N,K", [(1, 5, 128, 128), (4, 33, 200, 256), (8, 64, 256, 512), (7, 300, 136, 384),
                                        (64, 128, 256, 640), (60, 1000, 384, 272), (5, 1500, 264, 130), (130, 90, 128, 256),
                                        (3, 2000, 512, 1024), (1, 700, 256, 2048), (16, 16, 1100, 4096)])
def test_gemm_grouped(E, rows, N, K):
    rng = np.random.default_rng(E + rows + N)
    Kb, Nb = -(-K // 128), -(-N // 128)
    for kind, out, fa, align, spread in (("ints", "f32", "e4m3", 1, True), ("normal", "bf16", "e5m2", 1, False),
                                         ("ints", "f32", "e4m3", 1, False)):
        qa, sa = _bytes(rng, rows, K, fa, kind), _scale_of(rng, (Kb, rows), kind)
        qb, sb = _bytes(rng, E * N, K, "e4m3", kind), _scale_of(rng, (E, Nb, Kb), kind)
        off = _grouped_offsets(rng, E, rows, align)
        if not spread:
            off[0], off[-1] = 0, rows
        Kp = K + -K % 16
        B = fp8_dev(qb, "e4m3", Kp - K)
        B = B.as_strided((E, N, K), (N * Kp, Kp, 1))
        C = nm.fp8_gemm_nt_grouped(fp8_dev(qa, fa, Kp - K), dev(sa)[0], B, torch.from_numpy(sb).float().cuda(), i32(off),
                                   out_dtype=TD[out])
        a = MO.values_rows(qa, sa, fa)
        ref, mag = np.zeros((rows, N)), np.zeros((rows, N))
        for e in range(E):
            b = MO.values_blocks(qb[e * N:(e + 1) * N], sb[e], "e4m3")
            ref[off[e]:off[e + 1]], mag[off[e]:off[e + 1]] = _ref(a[off[e]:off[e + 1]], b)
        _check_product(host(C), ref, mag, out, kind, (kind, spread))


@pytest.mark.parametrize("E,M,N,rows", [(1, 128, 128, 128), (4, 130, 72, 640), (8, 256, 264, 1024), (60, 64, 200, 2048),
                                        (3, 300, 520, 4096)])
def test_gemm_grouped_k(E, M, N, rows):
    rng = np.random.default_rng(E + M + rows)
    for kind, out, fa in (("ints", "f32", "e4m3"), ("normal", "f32", "e5m2"), ("normal", "bf16", "e4m3")):
        qa, sa = _bytes(rng, M, rows, fa, kind), _scale_of(rng, (rows // 128, M), kind)
        qb, sb = _bytes(rng, N, rows, "e4m3", kind), _scale_of(rng, (rows // 128, N), kind)
        off = _grouped_offsets(rng, E, rows, 128)
        C = nm.fp8_gemm_nt_grouped_k(fp8_dev(qa, fa), dev(sa)[0], fp8_dev(qb, "e4m3"), dev(sb)[0], i32(off),
                                     out_dtype=TD[out])
        a, b = MO.values_rows(qa, sa, fa), MO.values_rows(qb, sb, "e4m3")
        for e in range(E):
            ref, mag = _ref(a[:, off[e]:off[e + 1]], b[:, off[e]:off[e + 1]])
            _check_product(host(C[e]), ref, mag, out, kind, (kind, out, e))


@pytest.mark.parametrize("K", [1024, 1168])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped_products_of_many_tiles(out, K):
    """Uneven groups over hundreds of workgroups, five times each: every repeat the exact integers (bf16:
    within its rounding) and the same bits."""
    rng = np.random.default_rng(K)
    E, N = 24, 640
    counts = rng.geometric(0.003, size=E)
    counts[3] = counts[11] = 0
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1]) + 100                                    # the last 100 rows belong to no group
    Kb, Nb = -(-K // 128), N // 128
    g = torch.Generator(device="cuda").manual_seed(K)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()
    power = lambda *s: torch.tensor([0.125, 0.25, 0.5, 1.0, 2.0, 4.0], device="cuda")[
        torch.randint(0, 6, s, generator=g, device="cuda")]
    a, b = ints(rows, K), ints(E, N, K)
    sa, sb = power(Kb, rows), power(E, Nb, Kb)
    wide = lambda s: s.repeat_interleave(128, -1)[..., :K].double()
    A = a.double() * wide(sa.t())
    ref = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
    for e in range(E):
        B = b[e].double() * wide(sb[e].repeat_interleave(128, 0))
        ref[off[e]:off[e + 1]] = A[off[e]:off[e + 1]] @ B.t()
    q = lambda x: x.to(torch.float8_e4m3fn)
    first = None
    for _ in range(5):
        C = nm.fp8_gemm_nt_grouped(q(a), sa, q(b), sb, i32(off), out_dtype=TD[out])
        first = C if first is None else first
        assert torch.equal(C, first)
    assert bool(((C.double() - ref).abs() <= (0 if out == "f32" else 2.0 ** -8) * ref.abs()).all())
    # the reduction grouped: runs of rows padded to 128
    up = np.concatenate([[0], np.cumsum(-(-counts // 128) * 128)]).astype(np.int32)
    R = int(up[-1])
    x, y = ints(700, R), ints(520, R)
    sx, sy = power(R // 128, 700), power(R // 128, 520)
    full = lambda s: s.t().repeat_interleave(128, 1).double()
    X, Y = x.double() * full(sx), y.double() * full(sy)
    first = None
    for _ in range(5):
        C = nm.fp8_gemm_nt_grouped_k(q(x), sx, q(y), sy, i32(up), out_dtype=TD[out])
        first = C if first is None else first
        assert torch.equal(C, first)
    for e in range(E):
        ref = X[:, up[e]:up[e + 1]] @ Y[:, up[e]:up[e + 1]].t()
        assert bool(((C[e].double() - ref).abs() <= (0 if out == "f32" else 2.0 ** -8) * ref.abs()).all())


# ---- combine ------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,D", [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (17, 8, 512), (5, 6, 1000), (9, 64, 64),
                                   (130, 5, 2056)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combine(T, k, D, dtype):
    rng = np.random.default_rng(T + k + D)
    for pad, shift in ((0, 0), (8, 0), (3, 0)):
        E = 16
        ids = rng.integers(-1, E, size=(T, k)).astype(np.int32)
        off, cnt, src, pos = MO.plan(ids, E, 16, nm.moe_plan_rows(T * k, E, 16))
        dO_, O = dev(rng.normal(size=(src.size, D)), dtype, pad)
        dw_, w = dev(rng.normal(size=(T, k)))
        dY_, dY = dev(rng.normal(size=(T, D)), dtype, pad)
        for weights in (dw_, None):
            y = MO.combine(O, pos, w if weights is not None else None)
            mag = MO.combine(np.abs(O), pos, np.abs(w) if weights is not None else None)
            got = host(nm.moe_combine(dO_, i32(pos), weights))
            assert (np.abs(got - y) <= 64 * 2.0 ** -24 * mag + half_ulp(y, dtype)).all()
        gO, gw = nm.moe_combine_bwd(dY_, dO_, i32(src), i32(pos), dw_)
        rO, rw = MO.combine_bwd(dY, O, pos, w)
        assert (np.abs(host(gO) - rO) <= 2.0 ** -23 * np.abs(rO) + half_ulp(rO, dtype)).all()
        live = pos >= 0
        magw = np.zeros((T, k))
        magw[live] = (np.abs(dY)[:, None] * np.abs(O)[np.maximum(pos, 0)]).sum(2)[live]
        assert (np.abs(host(gw) - rw) <= (D / 256 + 16) * 2.0 ** -23 * magw).all()
        assert (host(gw)[~live] == 0).all()


# ---- streams, repeats, graphs -------------------------------------------------------------------
def _layer_step():
    T, E, k, D, F = 96, 16, 4, 256, 384
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    wu, su = nm.fp8_quantize_weight((torch.randn(E, F, D, generator=g, device="cuda") * 0.05).bfloat16())
    wd, sd = nm.fp8_quantize_weight((torch.randn(E, D, F, generator=g, device="cuda") * 0.05).bfloat16())

    def step():
        ids, w = nm.moe_route(logits, k)
        off, cnt, src, pos = nm.moe_plan(ids, E, 128)
        q, s = nm.fp8_quantize(x, src=src, div=k)
        h = nm.fp8_gemm_nt_grouped(q, s, wu, su, off)
        hq, hs = nm.fp8_quantize(h, gate=h)
        o = nm.fp8_gemm_nt_grouped(hq, hs, wd, sd, off)
        return nm.moe_combine(o, pos, w), o, src, pos, w
    return step


def test_repeats_and_side_stream_are_identical():
    step = _layer_step()
    first = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = step()
    s.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_graph_replays_match_eager():
    step = _layer_step()
    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
