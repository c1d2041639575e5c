"""The mixture-of-experts FFN's operators in 8-bit floating point, as measured work.

Five operators, each in a plain form (elementary torch operations in 32 bits) and as the calls a
user makes of the framework:

  route     scores of a router -> experts, weights, the rows' order by expert, the scores' gradient
  quantize  rows (and columns) of 128-blocks to 8 bits with a power-of-two scale per block
  gemm      the product of two 8-bit matrices with a scale for each block of 128
  experts   the same product for every expert: rows grouped (forward, input gradient) or the
            reduction grouped (weight gradient)
  combine   the weighted sum of each token's expert rows, and its gradients

`listed()` are twelve cases, `draw(rng)` gives more of the same ranges.  Sizes are the framework's
FFN sizes (d_model 2048 and 4096, d_ff 8192 and 16384, 4096 and 8192 tokens) and generic expert
sizes (8 to 256 experts, up to 8 of them per token, expert width 1024).
"""

import math

import numpy as np
import torch

own = False

_FMT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _up(n, m):
    return (n + m - 1) // m * m


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # serving one token: 8 of 64 experts by softmax, and its 8 rows' order
        {"name": "route_one_token", "op": "route", "T": 1, "E": 64, "k": 8, "dtype": "bf16", "score": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "group_top": 2, "renorm": True, "scale": 1.0, "align": 1,
         "padding": 0, "train": False},
        # a training batch of 8192 tokens, the last 100 of them padding: sigmoid scores with a
        # balancing bias, 4 of 8 groups, 8 of 256 experts, rows padded to 128, and the gradient
        {"name": "route_train", "op": "route", "T": 8192, "E": 256, "k": 8, "dtype": "f32", "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "align": 128,
         "padding": 100, "train": True},
        # the hidden activations of 128 expert rows (16 tokens, 8 experts each): ReLU and 8 bits
        {"name": "quantize_relu_decode", "op": "quantize", "T": 128, "K": 1024, "k": 1, "E": 0, "dtype": "bf16",
         "fmt": "e4m3", "align": 1, "gate": True, "train": False},
        # 4096 tokens gathered into their 8 experts' rows, in the forward's rows and in the columns
        # the weight gradient reads
        {"name": "quantize_dispatch_train", "op": "quantize", "T": 4096, "K": 2048, "k": 8, "E": 64,
         "dtype": "bf16", "fmt": "e4m3", "align": 128, "gate": False, "train": True},
        # one token through the framework's 8192 x 2048 up-projection
        {"name": "gemm_one_token", "op": "gemm", "M": 1, "N": 8192, "K": 2048, "fa": "e4m3", "fb": "e4m3",
         "block": 128, "out": "bf16"},
        # the training step's up-projection: 8192 tokens, d_model 4096, d_ff 16384
        {"name": "gemm_up", "op": "gemm", "M": 8192, "N": 16384, "K": 4096, "fa": "e4m3", "fb": "e4m3",
         "block": 128, "out": "bf16"},
        # a weight gradient over 4096 tokens: both operands scaled along the tokens
        {"name": "gemm_wgrad", "op": "gemm", "M": 8192, "N": 2048, "K": 4096, "fa": "e5m2", "fb": "e4m3",
         "block": 1, "out": "f32"},
        # serving 16 tokens: 128 rows spread over 64 experts
        {"name": "experts_decode", "op": "experts", "T": 16, "k": 8, "E": 64, "N": 1024, "K": 2048, "fa": "e4m3",
         "out": "bf16", "align": 1, "by": "rows"},
        # a prompt of 4096 tokens, unevenly spread over the experts
        {"name": "experts_prefill", "op": "experts", "T": 4096, "k": 8, "E": 64, "N": 1024, "K": 2048, "fa": "e4m3",
         "out": "bf16", "align": 1, "by": "rows"},
        # the experts' weight gradients of 4096 tokens
        {"name": "experts_wgrad", "op": "experts", "T": 4096, "k": 8, "E": 64, "N": 2048, "K": 1024, "fa": "e5m2",
         "out": "f32", "align": 128, "by": "reduction"},
        # serving 16 tokens
        {"name": "combine_decode", "op": "combine", "T": 16, "k": 8, "E": 64, "D": 2048, "dtype": "bf16", "align": 1,
         "train": False},
        # a training batch, with the gradients of the rows and of the weights
        {"name": "combine_train", "op": "combine", "T": 8192, "k": 8, "E": 64, "D": 2048, "dtype": "bf16",
         "align": 128, "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "quantize", "gemm", "experts", "combine"])
    if op == "route":
        score = rng.choice(["softmax", "sigmoid"])
        train = rng.random() < 0.6
        T = _log(rng, 1, 8192)
        E = rng.choice([8, 16, 60, 64, 128, 160, 256])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 4])
        topk_groups = rng.randint(1, groups)
        k = min(rng.randint(1, 8), E // groups * topk_groups)
        return {"op": op, "T": T, "E": E, "k": k, "dtype": rng.choice(["bf16", "f32"]), "score": score,
                "bias": rng.random() < 0.5, "groups": groups, "topk_groups": topk_groups,
                "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5]),
                "align": rng.choice([1, 16, 128]), "padding": rng.choice([0, T // 50]), "train": train}
    if op == "quantize":
        train = rng.random() < 0.5
        k = rng.choice([1, 1, 2, 6, 8])
        T = _log(rng, 1, 32768 // k)
        K = rng.choice([_log(rng, 64, 2048), 128 * rng.randint(1, 16)])
        return {"op": op, "T": T, "K": K, "k": k, "E": 0 if k == 1 else rng.choice([8, 60, 64]),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "align": rng.choice([1, 16, 128]) if k > 1 else 1, "gate": rng.random() < 0.4, "train": train}
    if op == "gemm":
        while True:
            M = _log(rng, 1, 8192)
            N = rng.choice([_log(rng, 128, 16384), 128 * rng.randint(1, 128)])
            K = rng.choice([_log(rng, 128, 8192), 128 * rng.randint(1, 64), 128 * rng.randint(1, 64)])
            if M * N * K <= 8192 * 16384 * 4096:
                break
        block = rng.choice([128, 128, 1])
        return {"op": op, "M": M, "N": N, "K": K, "fa": rng.choice(["e4m3", "e5m2"]), "fb": "e4m3", "block": block,
                "out": rng.choice(["bf16", "f32"])}
    if op == "experts":
        by = rng.choice(["rows", "rows", "reduction"])
        E = rng.choice([8, 16, 60, 64, 128])
        k = rng.randint(1, 8)
        T = _log(rng, 1 if by == "rows" else 64, 4096)
        N = rng.choice([_log(rng, 128, 2048), 128 * rng.randint(1, 16)])
        K = rng.choice([_log(rng, 128, 2048), 128 * rng.randint(1, 16), 128 * rng.randint(1, 16)])
        return {"op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "fa": rng.choice(["e4m3", "e5m2"]),
                "out": rng.choice(["bf16", "f32"]), "align": 128 if by == "reduction" else rng.choice([1, 16, 128]),
                "by": by}
    k = rng.randint(1, 8)
    return {"op": op, "T": _log(rng, 1, 8192), "k": k, "E": rng.choice([8, 60, 64, 128]),
            "D": rng.choice([_log(rng, 64, 2048), 256 * rng.randint(1, 8)]), "dtype": rng.choice(["bf16", "f32"]),
            "align": rng.choice([1, 128]), "train": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _draw_ids(g, T, k, E):
    """k distinct experts per token, some experts more popular than others."""
    pop = torch.randn(E, generator=g, device="cuda") * 0.5
    noise = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    return torch.sort(pop - torch.log(-torch.log(noise)), dim=1, descending=True, stable=True)[1][:, :k].int().contiguous()


def _plan_plain(ids, E, align):
    """offsets [E + 1], counts [E], src [rows], pos [T, k] of the slots sorted by expert."""
    T, k = ids.shape
    n = T * k
    rows = _plan_rows(n, E, align)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    skey, order = torch.sort(key, stable=True)
    edges = torch.searchsorted(skey, torch.arange(E + 1, device=ids.device))
    counts = edges[1:] - edges[:-1]
    offsets = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    offsets[1:] = torch.cumsum((counts + align - 1) // align * align, 0)
    ext = torch.cat([offsets[:-1], offsets.new_full((1,), rows)])
    dest = ext[skey] + torch.arange(n, device=ids.device) - edges[skey]
    valid = skey < E
    dest = torch.where(valid, dest, torch.full_like(dest, rows))
    src = torch.full((rows + 1,), -1, dtype=torch.int32, device=ids.device)
    src[dest] = torch.where(valid, order, torch.full_like(order, -1)).int()
    pos = torch.empty(n, dtype=torch.int32, device=ids.device)
    pos[order] = torch.where(valid, dest, torch.full_like(dest, -1)).int()
    return offsets.int(), counts.int(), src[:rows].contiguous(), pos.view(T, k)


def _plan_rows(n, E, align):
    """Rows that T * k slots can take at most: every expert's segment is padded to `align`."""
    return _up(n + min(n, E) * (align - 1), align)


def _route_inputs(case, g):
    T, E = case["T"], case["E"]
    dt = _DT[case["dtype"]]
    bias = None
    if case["bias"]:
        # the balancing bias moves in steps of 0.001
        bias = torch.round(_normal(g, E, std=20.0)) * (1e-3 if case["score"] == "sigmoid" else 1e-4)
    logits = _normal(g, T, E, std=1.5, dtype=dt)
    # a choice that the last bits of a 32-bit score decide has no answer to compare: such rows are
    # drawn again (equal logits with equal biases stay: they go to the lowest index)
    for _ in range(12):
        close = _near_tie(case, logits, bias)
        n = int(close.sum())
        if n == 0:
            break
        logits[close] = _normal(g, n, E, std=1.5, dtype=dt)
    if case["padding"]:
        logits[T - case["padding"]:] = float("-inf")
    return logits, bias


def _near_tie(case, logits, bias):
    T, E = logits.shape
    l64 = logits.double()
    s = torch.softmax(l64, 1) if case["score"] == "softmax" else torch.sigmoid(l64)
    c = s if bias is None else s + bias.double()
    G = case["groups"]
    margin = 2e-6 * c.abs().amax(1, keepdim=True)
    close = torch.zeros(T, dtype=torch.bool, device=logits.device)
    if G > 1:
        gs = torch.sort(c.view(T, G, E // G), dim=2, descending=True)[0][:, :, :case["group_top"]].sum(2)
        v, i = torch.sort(gs, dim=1, descending=True, stable=True)
        close |= (v[:, :-1] - v[:, 1:] < 2 * margin).any(1)
        keep = torch.zeros(T, G, dtype=torch.bool, device=logits.device)
        keep.scatter_(1, i[:, :case["topk_groups"]], True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, torch.full_like(c, -1e30))
    v, i = torch.sort(c, dim=1, descending=True, stable=True)
    same = torch.gather(l64, 1, i[:, 1:]) == torch.gather(l64, 1, i[:, :-1])
    if bias is not None:
        same &= bias[i[:, 1:]] == bias[i[:, :-1]]
    gap = v[:, :-1] - v[:, 1:]
    return close | ((gap < margin) & ~same)[:, :case["k"]].any(1)


def _quantized(g, rows, K, fmt, std):
    """A random matrix in 8 bits with a scale per row and block of 128: q [rows, K] (its rows start at
    multiples of 128 bytes, as the quantizer leaves them), s [K / 128, rows]."""
    Kb = _up(K, 128) // 128
    x = torch.randn(rows, K, generator=g, device="cuda") * std
    x = torch.nn.functional.pad(x, (0, Kb * 128 - K)).view(rows, Kb, 128)
    s = x.abs().amax(2) / _MAX[fmt]
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (x / s.unsqueeze(2)).clamp_(-_MAX[fmt], _MAX[fmt]).to(_FMT[fmt]).view(rows, Kb * 128)
    return q[:, :K], s.t().contiguous()


def _quantized_blocks(g, E, N, K, fmt, std):
    """E random weights in 8 bits with a scale per 128 x 128 block: q [E, N, K] (rows as above),
    s [E, N / 128, K / 128]."""
    Nb, Kb = _up(N, 128) // 128, _up(K, 128) // 128
    q = torch.empty(E, N, Kb * 128, dtype=_FMT[fmt], device="cuda")
    s = torch.empty(E, Nb, Kb, device="cuda")
    for e in range(E):
        x = torch.randn(N, K, generator=g, device="cuda") * std
        x = torch.nn.functional.pad(x, (0, Kb * 128 - K, 0, Nb * 128 - N)).view(Nb, 128, Kb, 128)
        s[e] = x.abs().amax(3).amax(1) / _MAX[fmt]
        y = (x / s[e].view(Nb, 1, Kb, 1)).clamp_(-_MAX[fmt], _MAX[fmt])
        q[e] = y.view(Nb * 128, Kb * 128)[:N].to(_FMT[fmt])
    return q[:, :, :K], s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "route":
        st["logits"], st["bias"] = _route_inputs(case, g)
        if case["train"]:
            st["dweights"] = _normal(g, case["T"], case["k"])
    elif op == "quantize":
        T, K, k = case["T"], case["K"], case["k"]
        dt = _DT[case["dtype"]]
        # rows and columns of very different sizes, as activations are
        st["X"] = (torch.randn(T, K, generator=g, device="cuda") *
                   torch.exp(_normal(g, T, 1)) * torch.exp(_normal(g, 1, K, std=0.5))).to(dt)
        st["src"] = _plan_plain(_draw_ids(g, T, k, case["E"]), case["E"], case["align"])[2] if k > 1 else None
        # the gate of a row that is gathered belongs to its expert's row; else the row gates itself
        st["gate"] = None
        if case["gate"]:
            st["gate"] = st["X"] if k == 1 else _normal(g, st["src"].numel(), K, dtype=dt)
    elif op == "gemm":
        st["A"], st["sa"] = _quantized(g, case["M"], case["K"], case["fa"], 1.0)
        if case["block"] == 128:
            B, sb = _quantized_blocks(g, 1, case["N"], case["K"], case["fb"], 0.02)
            st["B"], st["sb"] = B[0], sb[0]
        else:
            st["B"], st["sb"] = _quantized(g, case["N"], case["K"], case["fb"], 1.0)
    elif op == "experts":
        ids = _draw_ids(g, case["T"], case["k"], case["E"])
        offsets, _, src, _ = _plan_plain(ids, case["E"], case["align"])
        st["offsets"], st["bounds"] = offsets, offsets.tolist()
        rows = src.numel()
        width = case["K"] if case["by"] == "rows" else case["N"]
        live = (src >= 0).float().unsqueeze(1)
        if case["by"] == "rows":
            st["A"], st["sa"] = _quantized(g, rows, width, case["fa"], 1.0)
            st["A"].copy_((st["A"].float() * live).to(st["A"].dtype))
            st["B"], st["sb"] = _quantized_blocks(g, case["E"], case["N"], case["K"], "e4m3", 0.02)
        else:
            st["A"], st["sa"] = _quantized(g, case["K"], rows, case["fa"], 0.01)
            st["B"], st["sb"] = _quantized(g, case["N"], rows, "e4m3", 1.0)
            for name in ("A", "B"):
                st[name].copy_((st[name].float() * live.t()).to(st[name].dtype))
    else:
        T, k, D = case["T"], case["k"], case["D"]
        dt = _DT[case["dtype"]]
        ids = _draw_ids(g, T, k, case["E"])
        _, _, st["src"], st["pos"] = _plan_plain(ids, case["E"], case["align"])
        st["O"] = _normal(g, st["src"].numel(), D, dtype=dt)
        w = torch.rand(T, k, generator=g, device="cuda") + 0.05
        st["weights"] = (w / w.sum(1, keepdim=True)).contiguous()
        if case["train"]:
            st["dY"] = _normal(g, T, D, dtype=dt)
    return st


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return (_RUN_OWN if own else _RUN)[case["op"]](case, state)


def _route_plain(case, st):
    logits, bias = st["logits"], st["bias"]
    T, E = logits.shape
    k, G, scale = case["k"], case["groups"], case["scale"]
    l = logits.float()
    ok = l > float("-inf")
    none = ~ok.any(1, keepdim=True)
    if case["score"] == "softmax":
        m = torch.where(none, torch.zeros_like(l[:, :1]), l.amax(1, keepdim=True))
        e = torch.where(ok, torch.exp(l - m), torch.zeros_like(l))
        s = e / torch.where(none, torch.ones_like(m), e.sum(1, keepdim=True))
    else:
        s = torch.where(ok, 1.0 / (1.0 + torch.exp(-l)), torch.zeros_like(l))
    low = torch.full_like(s, float("-inf"))
    c = torch.where(ok, s if bias is None else s + bias, low)
    if G > 1:
        top = torch.sort(c.view(T, G, E // G), dim=2, descending=True)[0][:, :, :case["group_top"]]
        # a group with fewer eligible experts than the score sums has the sum of those it has
        gs = torch.where((top > float("-inf")).any(2), torch.where(top > float("-inf"), top, torch.zeros_like(top)).sum(2),
                         torch.full_like(top[:, :, 0], float("-inf")))
        gi = torch.sort(gs, dim=1, descending=True, stable=True)[1][:, :case["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device)
        keep.scatter_(1, gi, True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, low)
    v, i = torch.sort(c, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    chosen = v > float("-inf")
    ids = torch.where(chosen, i, torch.full_like(i, -1)).int().contiguous()
    sj = torch.where(chosen, torch.gather(s, 1, i), torch.zeros_like(v))
    weights = sj
    if case["renorm"]:
        tot = sj.sum(1, keepdim=True)
        weights = sj / torch.where(tot > 0, tot, torch.ones_like(tot))
    weights = weights * scale
    out = [ids, weights, *_plan_plain(ids, E, case["align"])]
    if case["train"]:
        dw = st["dweights"] * chosen
        if case["renorm"]:
            ds = weights * (dw - (dw * weights).sum(1, keepdim=True) / scale)   # times s: ds_j s_j
        else:
            ds = weights * dw
        if case["score"] == "sigmoid":
            g = ds * (1.0 - sj)
            dl = torch.zeros_like(l).scatter_add_(1, i, g)
        else:
            dl = torch.zeros_like(l).scatter_add_(1, i, ds)
            if not case["renorm"]:
                dl = dl - s * ds.sum(1, keepdim=True)
        out.append(dl.to(logits.dtype))
    return out


def _route_own(case, st):
    import sparse_matmul_ffns_amd as nm
    kw = dict(score=case["score"], renorm=case["renorm"], scale=case["scale"])
    ids, weights = nm.moe_route(st["logits"], case["k"], bias=st["bias"], groups=case["groups"],
                                topk_groups=case["topk_groups"], group_top=case["group_top"], **kw)
    out = [ids, weights, *nm.moe_plan(ids, case["E"], align=case["align"])]
    if case["train"]:
        out.append(nm.moe_route_bwd(st["logits"], ids, weights, st["dweights"], **kw))
    return out


def _blocks_plain(x, fmt):
    """x [rows, blocks, 128] in 32 bits -> 8-bit values and the power-of-two scale of each block."""
    amax = x.abs().amax(2)
    mant, expo = torch.frexp(amax)
    # amax = mant * 2^expo with mant in [0.5, 1), the format's largest value 0.875 * 2^top: the
    # smallest power of two that is at least their quotient (and a normal number), from its exponent
    top = 9 if fmt == "e4m3" else 16
    expo = (expo - top + (mant > 0.875).int()).clamp(min=-126)
    s = torch.where(amax > 0, ((expo + 127) << 23).view(torch.float32), torch.ones_like(amax))
    return (x / s.unsqueeze(2)).to(_FMT[fmt]), s


def _quantize_plain(case, st):
    x = st["X"].float()
    if st["src"] is not None:
        src = st["src"].long()
        x = torch.where((src >= 0).unsqueeze(1), x[torch.div(src.clamp(min=0), case["k"], rounding_mode="floor")],
                        torch.zeros((), device=x.device))
    if st["gate"] is not None:
        x = torch.where(st["gate"].float() > 0, x, torch.zeros_like(x))
    R, K = x.shape
    Rp, Kp = _up(R, 128), _up(K, 128)
    q, s = _blocks_plain(torch.nn.functional.pad(x, (0, Kp - K)).view(R, Kp // 128, 128), case["fmt"])
    out = [q.view(R, Kp), s.t().contiguous()]
    if case["train"]:
        xt = torch.nn.functional.pad(x.t(), (0, Rp - R)).reshape(K, Rp // 128, 128)
        q, s = _blocks_plain(xt, case["fmt"])
        out += [q.view(K, Rp), s.t().contiguous()]
    return out


def _quantize_own(case, st):
    import sparse_matmul_ffns_amd as nm
    kw = dict(fmt=_FMT[case["fmt"]], src=st["src"], div=case["k"], gate=st["gate"])
    out = [*nm.fp8_quantize(st["X"], **kw)]
    if case["train"]:
        out += [*nm.fp8_quantize_t(st["X"], **kw)]
    return out


def _wide_rows(q, s):
    """The values of q [rows, K] with s [K / 128, rows]."""
    return q.float() * s.t().repeat_interleave(128, 1)[:, :q.shape[1]]


def _wide_blocks(q, s):
    """The values of q [N, K] with s [N / 128, K / 128]."""
    return q.float() * s.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def _gemm_plain(case, st):
    b = _wide_blocks(st["B"], st["sb"]) if case["block"] == 128 else _wide_rows(st["B"], st["sb"])
    return (_wide_rows(st["A"], st["sa"]) @ b.t()).to(_DT[case["out"]])


def _gemm_own(case, st):
    import sparse_matmul_ffns_amd as nm
    return nm.fp8_gemm_nt(st["A"], st["sa"], st["B"], st["sb"], b_block=case["block"], out_dtype=_DT[case["out"]])


def _experts_plain(case, st):
    bounds = st["bounds"]
    a = _wide_rows(st["A"], st["sa"])
    if case["by"] == "rows":
        out = torch.zeros(a.shape[0], case["N"], dtype=_DT[case["out"]], device="cuda")
        for e in range(case["E"]):
            if bounds[e + 1] > bounds[e]:
                out[bounds[e]:bounds[e + 1]] = (a[bounds[e]:bounds[e + 1]] @ _wide_blocks(st["B"][e], st["sb"][e]).t()
                                                ).to(out.dtype)
        return out
    b = _wide_rows(st["B"], st["sb"])
    out = torch.zeros(case["E"], case["K"], case["N"], dtype=_DT[case["out"]], device="cuda")
    for e in range(case["E"]):
        if bounds[e + 1] > bounds[e]:
            out[e] = (a[:, bounds[e]:bounds[e + 1]] @ b[:, bounds[e]:bounds[e + 1]].t()).to(out.dtype)
    return out


def _experts_own(case, st):
    import sparse_matmul_ffns_amd as nm
    call = nm.fp8_gemm_nt_grouped if case["by"] == "rows" else nm.fp8_gemm_nt_grouped_k
    return call(st["A"], st["sa"], st["B"], st["sb"], st["offsets"], out_dtype=_DT[case["out"]])


def _combine_plain(case, st):
    pos = st["pos"].long()
    O = st["O"].float()
    live = (pos >= 0).unsqueeze(2)
    picked = torch.where(live, O[pos.clamp(min=0)], torch.zeros((), device=O.device))
    w = st["weights"].unsqueeze(2)
    out = [(picked * w).sum(1).to(st["O"].dtype)]
    if case["train"]:
        dY = st["dY"].float()
        src = st["src"].long()
        slot = src.clamp(min=0)
        dO = dY[torch.div(slot, case["k"], rounding_mode="floor")] * st["weights"].reshape(-1)[slot].unsqueeze(1)
        out.append(torch.where((src >= 0).unsqueeze(1), dO, torch.zeros_like(dO)).to(st["O"].dtype))
        out.append((picked * dY.unsqueeze(1)).sum(2))
    return out


def _combine_own(case, st):
    import sparse_matmul_ffns_amd as nm
    out = [nm.moe_combine(st["O"], st["pos"], st["weights"])]
    if case["train"]:
        out += [*nm.moe_combine_bwd(st["dY"], st["O"], st["src"], st["pos"], st["weights"])]
    return out


_RUN = {"route": _route_plain, "quantize": _quantize_plain, "gemm": _gemm_plain, "experts": _experts_plain,
        "combine": _combine_plain}
_RUN_OWN = {"route": _route_own, "quantize": _quantize_own, "gemm": _gemm_own, "experts": _experts_own,
            "combine": _combine_own}


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    es = {"bf16": 2, "f32": 4}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b = T * E * es[case["dtype"]] + T * k * 12 + (2 * E + 1) * 4 + _plan_rows(T * k, E, case["align"]) * 4
        f = T * E * 8
        if case["train"]:
            b += T * E * es[case["dtype"]] + T * k * 4
            f += T * E * 4
        return {"bytes": b, "flops": f}
    if op == "quantize":
        R = case["T"] if case["k"] == 1 else _plan_rows(case["T"] * case["k"], case["E"], case["align"])
        K = case["K"]
        passes = 2 if case["train"] else 1
        b = case["T"] * K * es[case["dtype"]] + passes * (R * K + R * _up(K, 128) // 32)
        if case["k"] > 1:
            b += R * 4
            if case["gate"]:
                b += R * K * es[case["dtype"]]
        return {"bytes": b, "flops": 3 * passes * R * K}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        Kb = _up(K, 128) // 128
        sb = N * Kb if case["block"] == 1 else _up(N, 128) // 128 * Kb
        return {"bytes": M * K + N * K + 4 * (M * Kb + sb) + M * N * es[case["out"]], "flops": 2 * M * N * K}
    if op == "experts":
        n = case["T"] * case["k"]
        N, K = case["N"], case["K"]
        if case["by"] == "rows":
            # at least the experts of one token and at most all have a row: their weights are read
            live = min(case["E"], n)
            return {"bytes": n * K + live * N * K + n * N * es[case["out"]] + n * K // 32, "flops": 2 * n * N * K}
        return {"bytes": n * (N + K) + n * (N + K) // 32 + case["E"] * N * K * es[case["out"]],
                "flops": 2 * n * N * K}
    n, T, D = case["T"] * case["k"], case["T"], case["D"]
    e = es[case["dtype"]]
    b = n * D * e + T * D * e + n * 8
    f = 2 * n * D
    if case["train"]:
        b += T * D * e + n * D * e + n * 12
        f += 3 * n * D
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("gemm", "experts"):
        flops = work(case)["flops"]
        if flops > 4e12:
            return None
    return _EXACT[case["op"]](case, prepare(case, seed))


def _route_exact(case, st):
    l = st["logits"].double().cpu().numpy()
    bias = None if st["bias"] is None else st["bias"].double().cpu().numpy()
    T, E = l.shape
    k, G = case["k"], case["groups"]
    live = np.isfinite(l)
    lm = np.where(live, l, -np.inf)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if case["score"] == "softmax":
            top = np.where(live.any(1), lm.max(1), 0.0)[:, None]
            ex = np.exp(lm - top)
            s = ex / np.maximum(ex.sum(1, keepdims=True), 1e-300)
        else:
            s = np.where(live, 1.0 / (1.0 + np.exp(-lm)), 0.0)
    c = np.where(live, s + (0.0 if bias is None else bias[None, :]), -np.inf)
    index = np.arange(E)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    dl = np.zeros((T, E))
    dw = st["dweights"].double().cpu().numpy() if case["train"] else None
    for t in range(T):
        cand = live[t].copy()
        if G > 1:
            scores = []
            for q in range(G):
                part = np.sort(c[t, q * (E // G):(q + 1) * (E // G)])[::-1][:case["group_top"]]
                part = part[part > -np.inf]
                scores.append(part.sum() if part.size else -np.inf)
            best = np.lexsort((np.arange(G), -np.array(scores)))[:case["topk_groups"]]
            cand &= np.isin(index // (E // G), best)
        pick = index[cand]
        pick = pick[np.lexsort((pick, -c[t, pick]))][:k]
        n = pick.size
        if n == 0:
            continue
        ids[t, :n] = pick
        sj = s[t, pick]
        tot = sj.sum() if case["renorm"] else 1.0
        w[t, :n] = case["scale"] * sj / tot
        if dw is None:
            continue
        # through w_j = scale * s_j / (sum of the chosen s, or 1), then the scores' own derivative
        ds = np.zeros(E)
        ds[pick] = case["scale"] * dw[t, :n] / tot
        if case["renorm"]:
            ds[pick] -= case["scale"] * (dw[t, :n] * sj).sum() / tot ** 2
        dl[t] = s[t] * (ds - (ds * s[t]).sum()) if case["score"] == "softmax" else ds * s[t] * (1.0 - s[t])
    out = [torch.from_numpy(ids), torch.from_numpy(w)]
    align = case["align"]
    flat = ids.reshape(-1)
    rows = _plan_rows(flat.size, E, align)
    offsets, counts = np.zeros(E + 1, np.int32), np.zeros(E, np.int32)
    src, pos = np.full(rows, -1, np.int32), np.full(flat.size, -1, np.int32)
    for e in range(E):
        slots = np.nonzero(flat == e)[0]
        counts[e] = slots.size
        offsets[e + 1] = offsets[e] + -(-slots.size // align) * align
        src[offsets[e]:offsets[e] + slots.size] = slots
        pos[slots] = offsets[e] + np.arange(slots.size)
    out += [torch.from_numpy(a) for a in (offsets, counts, src, pos.reshape(T, k))]
    if case["train"]:
        out.append(torch.from_numpy(dl))
    return out


def _round8(y, fmt):
    """y (64 bits, within the format's range) rounded to the nearest 8-bit value, ties to even."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    expo = torch.frexp(y)[1] - 1
    step = _power(expo.clamp(min=low) - bits)
    return torch.round(y / step) * step


def _power(expo):
    """2^expo in 64 bits, exactly."""
    return ((expo.long() + 1023) << 52).view(torch.float64)


def _quantize_exact(case, st):
    x = st["X"].double()
    if st["src"] is not None:
        grown = torch.cat([x, torch.zeros_like(x[:1])])
        token = torch.where(st["src"] >= 0, st["src"] // case["k"], torch.full_like(st["src"], x.shape[0]))
        x = grown[token.long()]
    if st["gate"] is not None:
        x = x * (st["gate"] > 0)

    def along(y):
        n, m = y.shape
        full = torch.zeros(n, _up(m, 128), dtype=torch.float64, device=y.device)
        full[:, :m] = y
        part = full.view(n, -1, 128)
        peak = part.abs().max(2)[0]
        # near the quotient's logarithm, then stepped to the smallest power that is large enough
        power = _power(torch.log2(peak / _MAX[case["fmt"]]).ceil().clamp(min=-126))
        power = torch.where(power * _MAX[case["fmt"]] < peak, power * 2, power)
        power = torch.where(power * _MAX[case["fmt"]] >= 2 * peak, power / 2, power)
        power = torch.where(peak > 0, power, torch.ones_like(power))
        return [_round8(part / power.unsqueeze(2), case["fmt"]).view(n, -1), power.t().contiguous()]

    out = along(x)
    if case["train"]:
        out += along(x.t().contiguous())
    return out


def _values64(q, s, row_block):
    """The values of q [rows, K] in 64 bits; s per row (row_block 1, [K / 128, rows]) or per 128 x 128 block."""
    n, K = q.shape
    kb = torch.arange(K, device=q.device) // 128
    rb = torch.arange(n, device=q.device) // row_block
    s = s.double()
    return q.float().double() * (s[kb][:, rb].t() if row_block == 1 else s[rb][:, kb])


def _gemm_exact(case, st):
    return torch.matmul(_values64(st["A"], st["sa"], 1), _values64(st["B"], st["sb"], case["block"]).t())


def _experts_exact(case, st):
    edge = st["offsets"].tolist()
    if case["by"] == "rows":
        out = torch.zeros(st["A"].shape[0], case["N"], dtype=torch.float64, device="cuda")
        a = _values64(st["A"], st["sa"], 1)
        for e in range(case["E"]):
            if edge[e] < edge[e + 1]:
                out[edge[e]:edge[e + 1]] = torch.matmul(a[edge[e]:edge[e + 1]],
                                                        _values64(st["B"][e], st["sb"][e], 128).t())
        return out
    a, b = _values64(st["A"], st["sa"], 1), _values64(st["B"], st["sb"], 1)
    out = torch.zeros(case["E"], case["K"], case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        out[e] = torch.matmul(a[:, edge[e]:edge[e + 1]], b[:, edge[e]:edge[e + 1]].t())
    return out


def _combine_exact(case, st):
    T, k = st["pos"].shape
    w = st["weights"].double()
    O = st["O"].double()
    y = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    dO = torch.zeros_like(O) if case["train"] else None
    for j in range(k):
        p = st["pos"][:, j].long()
        t = torch.nonzero(p >= 0).squeeze(1)
        p = p[t]
        y[t] += w[t, j].unsqueeze(1) * O[p]
        if case["train"]:
            dY = st["dY"][t].double()
            dw[t, j] = (dY * O[p]).sum(1)
            dO[p] = w[t, j].unsqueeze(1) * dY
    return [y, dO, dw] if case["train"] else [y]


_EXACT = {"route": _route_exact, "quantize": _quantize_exact, "gemm": _gemm_exact, "experts": _experts_exact,
          "combine": _combine_exact}
