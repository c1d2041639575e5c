"""The mixture-of-experts FFN layer (moe.py) against the same layer in fp64 without quantisation.

Each operand in 8 bits carries a relative error of at most half a unit in the last place, 2^-4 for e4m3
and 2^-3 for e5m2, spread evenly: 0.036 and 0.072 root mean square.  Independent errors add in squares:
the output has four quantised operands in its chain (x, W_up, h, W_down), 0.072; the gradients two of
e5m2 and two to four of e4m3, 0.125.  The tests allow 1.5 times that in relative Frobenius norm.  ReLU's
derivative is taken where the layer's own pre-activations are positive: next to zero the 8-bit products
may have another sign than the reference's, and the gradient is that of the function that was computed.
"""

import numpy as np
import pytest
import torch

import sparse_matmul_ffns_amd as nm
from oracle import moe_oracle as MO
from sparse_matmul_ffns_amd.moe import ExpertFFN
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


@pytest.mark.parametrize("T,E,k,D,F,score", [(200, 8, 2, 256, 384, "softmax"), (1, 16, 4, 128, 256, "sigmoid"),
                                             (77, 6, 3, 200, 136, "sigmoid")])
def test_layer_forward_and_backward(T, E, k, D, F, score):
    rng = np.random.default_rng(T)
    bf = lambda *s, std=1.0: torch.from_numpy(rng.normal(size=s) * std).bfloat16()
    x, wu, wd, dy = bf(T, D), bf(E, F, D, std=D ** -0.5), bf(E, D, F, std=F ** -0.5), bf(T, D)
    logits = torch.from_numpy(rng.normal(size=(T, E))).float()
    if T > 1:
        logits[0] = -float("inf")        # a token of no expert
    f64 = lambda t: t.double().numpy()
    ids, w, _ = MO.route(f64(logits), k, score, scale=1.5)
    layer = ExpertFFN(wu.cuda(), wd.cuda(), k, score=score, scale=1.5, train=True)
    y = layer.forward(x.cuda(), logits.cuda())
    pos, pre = layer.saved[6].cpu().numpy(), f64(layer.saved[7].cpu())
    X, U, W, G = f64(x), f64(wu), f64(wd), f64(dy)
    Y, dX = np.zeros((T, D)), np.zeros((T, D))
    dU, dD, dw = np.zeros(U.shape), np.zeros(W.shape), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            h = U[e] @ X[t]
            a = np.maximum(h, 0)
            o = W[e] @ a
            Y[t] += w[t, j] * o
            dw[t, j] = G[t] @ o
            do = w[t, j] * G[t]
            dh = (W[e].T @ do) * (pre[pos[t, j]] > 0)
            dD[e] += np.outer(do, a)
            dU[e] += np.outer(dh, X[t])
            dX[t] += U[e].T @ dh
    dl = MO.route_bwd(f64(logits), ids, w, dw, score, True, 1.5)
    got = layer.backward(dy.cuda())
    assert _rel(f64(y.cpu()), Y) < 1.5 * 0.072
    for g, ref, name in zip(got, (dX, dl, dU, dD), ("dx", "dlogits", "dW_up", "dW_down")):
        g = f64(g.cpu())
        assert g.shape == ref.shape and _rel(g, ref) < 1.5 * 0.125, (name, _rel(g, ref))
    if T > 1:
        assert (f64(y.cpu())[0] == 0).all() and (f64(got[0].cpu())[0] == 0).all() and (f64(got[1].cpu())[0] == 0).all()
    # serving: no padding between the experts' rows, the same products
    serve = ExpertFFN(wu.cuda(), wd.cuda(), k, score=score, scale=1.5)
    assert torch.equal(serve.forward(x.cuda(), logits.cuda()), y)
    with pytest.raises(RuntimeError):
        serve.backward(dy.cuda())


def test_exported():
    assert nm.ExpertFFN is ExpertFFN
