"""The dense FFN block (dense.py) against the same block in fp64 on the same bf16 weights.

The block rounds to bf16 (relative 2^-8 at most, 2^-8 / sqrt(3) root mean square: 0.0023) its norm's output, its activations,
its pre-activations, the gradient between the products and what leaves it.  Independent errors add in squares: the
output carries three of them in its FFN part, a gradient at most six (0.0055); the tests allow 1.5 times that in relative Frobenius
norm.  The gradients are also held to differences of a 64-bit block.
"""

import threading

import numpy as np
import pytest
import torch

import sparse_matmul_ffns_amd as nm
from oracle import dense_oracle as O
from sparse_matmul_ffns_amd import DenseFFN
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
LIMIT = 1.5 * 0.0055


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _rel(a, b):
    a = a.detach().double().cpu().numpy()
    return np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-30)


def _parts(T, D, F, act, bias, seed):
    rng = np.random.default_rng(seed)
    bf = lambda *s, std=1.0: torch.from_numpy(rng.normal(size=s) * std).bfloat16()
    return dict(x=bf(T, D), r=bf(T, D), wn=1 + bf(D, std=0.2), wu=bf(F, D, std=D ** -0.5), wd=bf(D, F, std=F ** -0.5),
                bu=bf(F, std=0.3) if bias else None, bd=bf(D, std=0.3) if bias else None, dy=bf(T, D))


def _block64(p, act):
    """(y, gradients) in 64 bits: dx, w_norm, W_up, W_down, b_up, b_down."""
    f = {k: None if v is None else v.double().numpy() for k, v in p.items()}
    n, h, rstd = O.rms_norm(f["x"], f["wn"], 1e-5, f["r"])
    a, z = O.linear(n, f["wu"], f["bu"], act)
    y = O.linear(a, f["wd"], f["bd"], "none", h)[0]
    dz = (f["dy"] @ f["wd"]) * O.dact(z, act)
    dx, dw = O.rms_norm_bwd(dz @ f["wu"], h, f["wn"], rstd, f["dy"])
    return y, [dx, dw, dz.T @ n, f["dy"].T @ a, dz.sum(0), f["dy"].sum(0)]


def _layer(p, act, train=True):
    c = lambda t: None if t is None else t.cuda()
    return DenseFFN(c(p["wn"]), c(p["wu"]), c(p["wd"]), c(p["bu"]), c(p["bd"]), act=act, train=train)


@pytest.mark.parametrize("T,D,F,bias", [(200, 256, 512, True), (1, 128, 384, True), (77, 200, 136, False), (65, 111, 257, True),
                                        (600, 512, 2048, True)])
@pytest.mark.parametrize("act", ["gelu_tanh", "relu", "silu", "none"])
def test_forward_and_backward(T, D, F, bias, act):
    p = _parts(T, D, F, act, bias, T + D)
    y64, g64 = _block64(p, act)
    layer = _layer(p, act)
    y = layer.forward(p["x"].cuda(), p["r"].cuda())
    h64 = (p["x"].double() + p["r"].double()).numpy()
    assert np.linalg.norm(y.double().cpu().numpy() - y64) <= LIMIT * np.linalg.norm(y64)
    # ReLU's kink: next to zero the rounded pre-activation may lie on the other side; those few entries change a gradient
    # by their whole size, so the gradients of 'relu' are compared at the layer's own activations
    if act == "relu":
        f = {k: None if v is None else v.double().numpy() for k, v in p.items()}
        n, h, rstd = O.rms_norm(f["x"], f["wn"], 1e-5, f["r"])
        a = layer.saved[4].double().cpu().numpy()
        dz = (f["dy"] @ f["wd"]) * (a > 0)
        dx, dw = O.rms_norm_bwd(dz @ f["wu"], h, f["wn"], rstd, f["dy"])
        g64 = [dx, dw, dz.T @ n, f["dy"].T @ a, dz.sum(0), f["dy"].sum(0)]
    dx, grads = layer.backward(p["dy"].cuda())
    got = [dx, *grads]
    assert len(got) == (6 if bias else 4)
    for name, a, b in zip(("dx", "w_norm", "W_up", "W_down", "b_up", "b_down"), got, g64):
        assert a.dtype == (torch.bfloat16 if name == "dx" else torch.float32) and a.shape == b.shape
        assert _rel(a, b) <= LIMIT, (name, _rel(a, b))
    assert h64.shape == y64.shape
    # a layer that does not train gives the same
    assert torch.equal(_layer(p, act, train=False).forward(p["x"].cuda(), p["r"].cuda()), y)
    # without a residual
    y2 = layer.forward((p["x"].double() + p["r"].double()).bfloat16().cuda())
    assert _rel(y2, y64) <= LIMIT


def test_gradients_against_differences():
    """The block's loss sum(y dy), in 64 bits, moves by the gradient times the step in random directions."""
    p = _parts(40, 64, 96, "gelu_tanh", True, 3)
    dx, grads = (lambda l: (l.forward(p["x"].cuda(), p["r"].cuda()), l.backward(p["dy"].cuda()))[1])(_layer(p, "gelu_tanh"))
    rng = np.random.default_rng(4)
    for key, g in zip(("x", "wn", "wu", "wd", "bu", "bd"), (dx, *grads)):
        d = torch.from_numpy(rng.normal(size=p[key].shape))
        loss = []
        for sign in (1, -1):
            q = dict(p, **{key: p[key].double() + sign * 1e-4 * d})
            loss.append((_block64(q, "gelu_tanh")[0] * p["dy"].double().numpy()).sum())
        want = (loss[0] - loss[1]) / 2e-4
        terms = (g.double().cpu() * d).numpy()
        # independent relative errors of LIMIT in the terms, at four times their root of squares
        assert abs(terms.sum() - want) <= 4 * LIMIT * np.sqrt((terms ** 2).sum()) + 1e-4 * abs(want), key


def test_passes_and_clipping():
    ps = [_parts(50 + 3 * i, 128, 256, "silu", True, i) for i in range(3)]
    layer = _layer(ps[0], "silu")
    for p in ps[1:]:
        p.update({k: ps[0][k] for k in ("wn", "wu", "wd", "bu", "bd")})
    waiting = [layer.forward(p["x"].cuda(), p["r"].cuda(), return_saved=True)[1] for p in ps]
    for p, saved in reversed(list(zip(ps, waiting))):
        dx, grads = layer.backward(p["dy"].cuda(), saved)
        _, g64 = _block64(p, "silu")
        assert _rel(dx, g64[0]) <= LIMIT and all(_rel(a, b) <= LIMIT for a, b in zip(grads, g64[1:]))
    want = np.sqrt(sum((g.double() ** 2).sum().item() for g in grads))
    keep = [g.clone() for g in grads]
    norm = nm.grad_clip(grads, want / 4)
    assert abs(float(norm) - want) <= 1e-6 * want
    assert all(torch.allclose(a, b / 4, rtol=1e-6, atol=0) for a, b in zip(grads, keep))
    # lost passes and changed inputs
    x = ps[0]["x"].cuda()
    layer.forward(x)
    layer.forward(x)
    layer.backward(x)
    with pytest.raises(RuntimeError):
        layer.backward(x)
    layer.forward(x)
    x.add_(1)
    with pytest.raises(RuntimeError):
        layer.backward(x)
    layer.forward(x)
    layer.W_up.mul_(2)
    with pytest.raises(RuntimeError):
        layer.backward(x)


def test_threads_on_streams_of_their_own():
    """One layer, four threads with a stream each, passes of different sizes at once: each gives what it gives alone."""
    ps = [_parts(60 + 70 * i, 256, 520, "silu", True, i) for i in range(4)]
    for p in ps[1:]:
        p.update({k: ps[0][k] for k in ("wn", "wu", "wd", "bu", "bd")})
    layer = _layer(ps[0], "silu")
    args = [[p[k].cuda() for k in ("x", "r", "dy")] for p in ps]

    def step(x, r, dy):
        y, saved = layer.forward(x, r, return_saved=True)
        dx, grads = layer.backward(dy, saved)
        return [y, dx, nm.grad_clip(grads, 0.1), *grads]
    want = [step(*a) for a in args]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(10):
                    got[i] = step(*args[i])
            stream.synchronize()
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_the_layer_in_a_graph():
    """A training step captured once and replayed with new inputs and weights, an eager step between the replays."""
    p = _parts(130, 128, 264, "gelu_tanh", True, 9)
    layer = _layer(p, "gelu_tanh")
    x, r, dy = (p[k].cuda() for k in ("x", "r", "dy"))

    def step():
        y, saved = layer.forward(x, r, return_saved=True)
        dx, grads = layer.backward(dy, saved)
        return [y, dx, nm.grad_clip(grads, 0.1), *grads]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.mul_(-0.5)
        layer.W_up.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), i


def test_the_norm_feeds_the_8_bit_product():
    """rms_norm_fp8's result as fp8_gemm_nt takes it, against the 64-bit norm and product: two operands of half a
    step of e4m3 each (0.036 root mean square), and the bf16 result."""
    rng = np.random.default_rng(8)
    T, D, N = 130, 520, 256
    x, r, w = (torch.from_numpy(rng.normal(size=s)).bfloat16() for s in ((T, D), (T, D), (N, D)))
    wn = torch.from_numpy(1 + 0.1 * rng.normal(size=D)).float()
    q, s, h, _ = nm.rms_norm_fp8(x.cuda(), wn.cuda(), residual=r.cuda())
    qw, sw = nm.fp8_quantize_weight(w.cuda())
    y = nm.fp8_gemm_nt(q[:, :D], s, qw[:, :D], sw)
    want = O.rms_norm(x.double().numpy(), wn.double().numpy(), 1e-5, r.double().numpy())[0] @ w.double().numpy().T
    assert _rel(y, want) <= 1.5 * np.sqrt(2) * 0.036
