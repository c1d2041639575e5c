"""fp64 oracle of the mixture-of-experts FFN in 8-bit floating point (CPU, numpy).

Written from the definitions alone; shares no code with the library.  Raw inputs are float64 arrays
of values that the device holds exactly (bf16 or fp32), 8-bit matrices are uint8 bytes.
"""

from __future__ import annotations

import numpy as np

MAX8 = {"e4m3": 448.0, "e5m2": 57344.0}
NEG = -np.inf


def decode8(fmt: str) -> np.ndarray:
    """The value of each of the 256 bytes, from the formats' definition (OCP: e4m3 has no infinity and
    NaN at 0x7F / 0xFF; e5m2 has infinity at 0x7C and NaN above)."""
    out = np.empty(256)
    man, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    for b in range(256):
        s, e, m = b >> 7, (b & 0x7F) >> man, b & ((1 << man) - 1)
        if e == 0:
            v = m * 2.0 ** (1 - bias - man)
        else:
            v = (1 + m / 2 ** man) * 2.0 ** (e - bias)
        if fmt == "e4m3" and (b & 0x7F) == 0x7F:
            v = np.nan
        if fmt == "e5m2" and e == 31:
            v = np.inf if m == 0 else np.nan
        out[b] = -v if s else v
    return out


def encode8(y: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest byte to each value, ties to the even significand; NaN (and infinities) to NaN's byte."""
    vals = decode8(fmt)[:128]
    fin = vals[np.isfinite(vals)]            # ascending
    a = np.abs(y)
    bad = ~np.isfinite(a)
    a = np.where(bad, 0.0, a)
    assert (a <= fin[-1]).all()
    hi = np.searchsorted(fin, a)             # first >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - fin[lo], fin[hi] - a
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == fin[hi], hi, code).astype(np.uint8)
    code = code | np.where(np.signbit(y), 0x80, 0).astype(np.uint8)
    return np.where(bad, np.uint8(0x7F), code)


def block_scale(block: np.ndarray, fmt: str) -> float:
    """The smallest power of two, at least 2^-126, that is >= the largest finite magnitude / max; 1 for 0."""
    fin = np.abs(block[np.isfinite(block)])
    amax = fin.max() if fin.size else 0.0
    if amax == 0.0:
        return 1.0
    e = -126
    while 2.0 ** e * MAX8[fmt] < amax:
        e += 1
    return 2.0 ** e


def rows_of(x, src=None, div=1, gate=None):
    """The quantisers' input: gathered rows, then the gate."""
    if src is not None:
        out = np.zeros((len(src), x.shape[1]))
        for r, s in enumerate(src):
            if s >= 0 and s // div < x.shape[0]:
                out[r] = x[s // div]
        x = out
    if gate is not None:
        x = np.where(gate > 0, x, 0.0)
    return x


def quantize(x, fmt):
    """Rows: bytes [R, Kp], scales [Kp / 128, R]."""
    R, K = x.shape
    Kb = -(-K // 128)
    p = np.zeros((R, Kb * 128))
    p[:, :K] = x
    s = np.ones((Kb, R))
    q = np.zeros(p.shape, np.uint8)
    for r in range(R):
        for b in range(Kb):
            blk = p[r, b * 128:(b + 1) * 128]
            s[b, r] = block_scale(blk, fmt)
            q[r, b * 128:(b + 1) * 128] = encode8(blk / s[b, r], fmt)
    return q, s


def quantize_weight(w, fmt):
    """One weight [N, K]: bytes [N, Kp], scales [N / 128, K / 128]."""
    N, K = w.shape
    Nb, Kb = -(-N // 128), -(-K // 128)
    q = np.zeros((N, Kb * 128), np.uint8)
    s = np.ones((Nb, Kb))
    for i in range(Nb):
        for j in range(Kb):
            blk = w[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
            s[i, j] = block_scale(blk, fmt)
            q[i * 128:i * 128 + blk.shape[0], j * 128:j * 128 + blk.shape[1]] = encode8(blk / s[i, j], fmt)
    return q, s


def values_rows(q, s, fmt):
    """Values of bytes q [R, K] with scales s [K / 128, R]."""
    return decode8(fmt)[q] * np.repeat(s.T, 128, axis=1)[:, :q.shape[1]]


def values_blocks(q, s, fmt):
    """Values of bytes q [N, K] with scales s [N / 128, K / 128]."""
    full = np.repeat(np.repeat(s, 128, axis=0), 128, axis=1)
    return decode8(fmt)[q] * full[:q.shape[0], :q.shape[1]]


def route(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=2, renorm=True, scale=1.0):
    """ids [T, k], weights [T, k] and the scores s [T, E]."""
    T, E = logits.shape
    l = np.where(np.isnan(logits), NEG, np.minimum(logits, np.finfo(np.float32).max))
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    S = np.zeros((T, E))
    for t in range(T):
        ok = l[t] > NEG
        if score == "softmax":
            top = l[t].max() if ok.any() else 0.0
            e = np.where(ok, np.exp(np.maximum(l[t] - top, -745.0)) * (l[t] - top > -745.0), 0.0)
            s = e / e.sum() if ok.any() else e
        else:
            with np.errstate(over="ignore"):
                s = np.where(ok, 1.0 / (1.0 + np.exp(-l[t])), 0.0)
        S[t] = s
        c = s if bias is None else s + bias
        # without a bias the order of the scores is that of the logits, which do not collapse
        order = l[t] if bias is None else c
        ok = ok & ~np.isnan(c) & (c > NEG)
        if groups > 1:
            n = E // groups
            sc = []
            for g in range(groups):
                best = sorted((c[e] for e in range(g * n, (g + 1) * n) if ok[e]), reverse=True)[:group_top]
                sc.append(sum(best) if best else NEG)
            keep = sorted(range(groups), key=lambda g: (-sc[g], g))[:topk_groups]
            ok = ok & np.array([e // n in keep for e in range(E)])
        pick = sorted((e for e in range(E) if ok[e]), key=lambda e: (-order[e], e))[:k]
        if not pick:
            continue
        ids[t, :len(pick)] = pick
        if renorm:
            if score == "softmax":
                r = np.exp(l[t, pick] - l[t, pick].max())
            else:
                m = np.minimum(l[t, pick], 0.0)
                r = np.exp(m - m.max()) / (1.0 + np.exp(-np.abs(l[t, pick])))
            w[t, :len(pick)] = scale * r / r.sum()
        else:
            w[t, :len(pick)] = scale * s[pick]
    return ids, w, S


def route_weights_of(logits, ids, score, renorm, scale):
    """The weights as a smooth function of the logits for a fixed choice."""
    out = np.zeros(ids.shape)
    for t in range(ids.shape[0]):
        if score == "softmax":
            e = np.exp(logits[t] - logits[t].max())
            s = e / e.sum()
        else:
            s = 1.0 / (1.0 + np.exp(-logits[t]))
        sel = ids[t] >= 0
        v = s[ids[t][sel]]
        out[t, sel] = scale * v / (v.sum() if renorm else 1.0)
    return out


def route_bwd(logits, ids, weights, dweights, score, renorm, scale):
    """dlogits [T, E] by the chain rule through the scores."""
    T, E = logits.shape
    dl = np.zeros((T, E))
    for t in range(T):
        fin = logits[t] > NEG
        sel = ids[t] >= 0
        if not sel.any():
            continue
        pick, dw = ids[t][sel], dweights[t][sel]
        if score == "softmax":
            e = np.where(fin, np.exp(np.where(fin, logits[t], 0.0) - logits[t][fin].max()), 0.0)
            s = e / e.sum()
        else:
            s = np.where(fin, 1.0 / (1.0 + np.exp(-np.where(fin, logits[t], 0.0))), 0.0)
        tot = s[pick].sum() if renorm else 1.0
        ds = np.zeros(E)
        ds[pick] = scale * dw / tot
        if renorm:
            ds[pick] -= scale * (dw * s[pick]).sum() / tot ** 2
        if score == "softmax":
            # sum_j ds_j s_j is 0 by definition where the weights are renormalised
            dl[t] = s * ds if renorm else s * (ds - (ds * s).sum())
        else:
            dl[t] = ds * s * (1.0 - s)
    return dl


def plan(ids, E, align, rows):
    flat = ids.reshape(-1)
    offsets, counts = np.zeros(E + 1, np.int32), np.zeros(E, np.int32)
    src, pos = np.full(rows, -1, np.int32), np.full(flat.size, -1, np.int32)
    for e in range(E):
        slots = np.nonzero(flat == e)[0]
        counts[e] = slots.size
        offsets[e + 1] = offsets[e] + -(-slots.size // align) * align
        src[offsets[e]:offsets[e] + slots.size] = slots
        pos[slots] = offsets[e] + np.arange(slots.size)
    return offsets, counts, src, pos.reshape(ids.shape)


def combine(O, pos, w):
    T, k = pos.shape
    y = np.zeros((T, O.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < O.shape[0]:
                y[t] += (1.0 if w is None else w[t, j]) * O[pos[t, j]]
    return y


def combine_bwd(dY, O, pos, w):
    T, k = pos.shape
    dO, dw = np.zeros(O.shape), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < O.shape[0]:
                dO[pos[t, j]] = w[t, j] * dY[t]
                dw[t, j] = (dY[t] * O[pos[t, j]]).sum()
    return dO, dw
