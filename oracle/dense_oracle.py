"""The dense FFN block's operators in fp64 on the CPU (numpy), with the worst error that fp32 arithmetic may make.

Plain definitions, independent of the library.  Every function takes and returns float64 arrays that hold the
operands' exact values.
"""

import math

import numpy as np

U = 2.0 ** -24          # half a step of fp32, relative
CUBE, GK = 0.044715, math.sqrt(2.0 / math.pi)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def act(z, kind):
    if kind == "relu":
        return np.where(z > 0, z, 0.0)
    if kind == "gelu_tanh":
        return z * sigmoid(2 * GK * (z + CUBE * z ** 3))
    if kind == "silu":
        return z * sigmoid(z)
    return z


def dact(z, kind):
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu_tanh":
        s = sigmoid(2 * GK * (z + CUBE * z ** 3))
        return s + z * s * (1 - s) * 2 * GK * (1 + 3 * CUBE * z * z)
    if kind == "silu":
        s = sigmoid(z)
        return s + z * s * (1 - s)
    return np.ones_like(z)


def _arg(z, kind):
    return 2 * GK * (z + CUBE * z ** 3) if kind == "gelu_tanh" else z


def act_error(z, kind):
    """What fp32 may be off by in act(z) for an exact z: the exponential's argument carries four roundings, and the
    exponential, the sum, the reciprocal and the product one each at one or two units: relative (8 |x| + 8) U."""
    if kind in ("none", "relu"):
        return np.zeros_like(z)
    x = np.minimum(np.abs(_arg(z, kind)), 200.0)
    return np.abs(act(z, kind)) * (8 * x + 8) * U + 1e-36


def dact_error(z, kind):
    """The same for the derivative s + z q s (1 - s): the relative error of s enters both terms, and 1 - s is off
    by a few U in itself.  Beyond |x| = 40 the sigmoid is 0 or 1 to the last bit that counts."""
    if kind in ("none", "relu"):
        return np.zeros_like(z)
    x = np.abs(_arg(z, kind))
    q = 2 * GK * (1 + 3 * CUBE * z * z) if kind == "gelu_tanh" else np.ones_like(z)
    near = 16 * U * (1 + np.minimum(x, 40)) * (1 + np.abs(z) * q)
    return np.where(x > 40, 4 * U, near)


def rms_norm(x, w, eps, residual=None):
    """(y, h, rstd)."""
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, h, rstd


def rms_norm_bwd(dy, h, w, rstd, dh=None):
    """(dx, dw) for an rstd that is given."""
    xh = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    return dx if dh is None else dx + dh, (dy * xh).sum(0)


def scales(y, fmt):
    """The power-of-two scale of each block of 128 columns [blocks, rows], and whether its largest magnitude lies so
    near a scale's border (1e-5) that fp32 may take the next one."""
    rows, cols = y.shape
    kb = -(-cols // 128)
    full = np.zeros((rows, kb * 128))
    full[:, :cols] = y
    amax = np.abs(full.reshape(rows, kb, 128)).max(2)
    q = amax / (448.0 if fmt == "e4m3" else 57344.0)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.ceil(np.log2(np.where(amax > 0, q, 1.0))), 0.0)
    e = np.maximum(e, -126)
    e = np.where((amax > 0) & (2.0 ** e < q), e + 1, e)
    m = q / 2.0 ** e                  # in (0.5, 1]
    near = (amax > 0) & ((m > 1 - 1e-5) | (m < 0.5 * (1 + 1e-5)))
    return (2.0 ** e).T, near.T


def linear(x, w, bias=None, kind="none", residual=None):
    """(y, z)."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(z, kind)
    return (y if residual is None else y + residual), z


def grad_norm(gs):
    return math.sqrt(math.fsum(float((g.astype(np.float64) ** 2).sum()) for g in gs))


def grad_factor(norm, max_norm):
    return max_norm / norm if max_norm < norm < math.inf else 1.0
