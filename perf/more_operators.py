"""The dense FFN block's operators around and in place of the sparse products, as measured work.

Three operators, each in a plain form (elementary torch operations in 32 bits) and as the calls a
user makes of the framework:

  norm    the residual's addition and the root-mean-square norm, its result in the input's type or in
          8 bits with a power-of-two scale per block of 128, and the gradients
  linear  the product of activations and a weight with bias, activation and residual in its epilogue;
          the activation's gradient and the bias's; the products of the backward pass
  clip    the norm of all gradients together, and the gradients scaled down to a largest norm

`listed()` are twelve cases, `draw(rng)` gives more of the same ranges.  Sizes are the framework's FFN
sizes (d_model 2048 and 4096, d_ff 8192 and 16384, 4096 and 8192 tokens), its experts' (64 of 1024 x
2048) and odd ones.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_TOP = {"e4m3": 448.0, "e5m2": 57344.0}
_ACTS = ["none", "relu", "gelu_tanh", "silu"]
_EPS = 1e-5


def _up(n, m):
    return (n + m - 1) // m * m


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # serving one token: the block's output joins the residual and is normed for the next product
        {"name": "norm_one_token", "op": "norm", "T": 1, "D": 4096, "dtype": "bf16", "wdtype": "bf16",
         "residual": True, "out": "same", "train": False},
        # a prompt of 4096 tokens, normed straight into the 8-bit product's operand
        {"name": "norm_prompt_8bit", "op": "norm", "T": 4096, "D": 2048, "dtype": "bf16", "wdtype": "bf16",
         "residual": True, "out": "e4m3", "train": False},
        # a training batch: forward, and the gradients with the one that comes through the residual
        {"name": "norm_train", "op": "norm", "T": 8192, "D": 4096, "dtype": "bf16", "wdtype": "f32",
         "residual": True, "out": "same", "train": True},
        # an odd width in 32 bits, without a residual
        {"name": "norm_odd_train", "op": "norm", "T": 999, "D": 1111, "dtype": "f32", "wdtype": "f32",
         "residual": False, "out": "same", "train": True},
        # serving one token through the 8192 x 2048 up-projection
        {"name": "linear_one_token", "op": "linear", "mode": "forward", "M": 1, "N": 8192, "K": 2048, "act": "relu",
         "bias": True, "residual": False, "pre": False, "out": "bf16"},
        # the training step's up-projection (8192 tokens, d_model 4096, d_ff 16384), which keeps the
        # pre-activations for the backward pass
        {"name": "linear_up_train", "op": "linear", "mode": "forward", "M": 8192, "N": 16384, "K": 4096,
         "act": "gelu_tanh", "bias": True, "residual": False, "pre": True, "out": "bf16"},
        # the down-projection of a prompt of 4096 tokens, added to the residual
        {"name": "linear_down", "op": "linear", "mode": "forward", "M": 4096, "N": 2048, "K": 8192, "act": "none",
         "bias": True, "residual": True, "pre": False, "out": "bf16"},
        # the gradient of a down-projection's output: through its weight and the ReLU before it, and the
        # weight's own (4096 tokens, d_ff 8192, d_model 2048)
        {"name": "linear_gradients", "op": "linear", "mode": "products", "M": 4096, "N": 2048, "K": 8192, "act": "relu",
         "out": "bf16"},
        # the gradient of an activation by itself, and the bias's
        {"name": "linear_act_gradient", "op": "linear", "mode": "act", "M": 4096, "N": 8192, "act": "gelu_tanh"},
        # a small module's gradients: a few matrices and vectors, where launches count
        {"name": "clip_small", "op": "clip", "matrices": 2, "rows": 128, "cols": 128, "vectors": 3, "odd": 1,
         "dtype": "f32", "out": "f32", "ratio": 0.5},
        # an FFN block of d_model 4096 and d_ff 16384: two weights, biases and the norm
        {"name": "clip_block", "op": "clip", "matrices": 2, "rows": 16384, "cols": 4096, "vectors": 3, "odd": 0,
         "dtype": "f32", "out": "f32", "ratio": 0.1},
        # 64 experts' weights, a tensor each, in 16 bits to the optimizer's 32
        {"name": "clip_experts", "op": "clip", "matrices": 128, "rows": 1024, "cols": 2048, "vectors": 64, "odd": 7,
         "dtype": "bf16", "out": "f32", "ratio": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "clip"])
    if op == "norm":
        out = rng.choice(["same", "same", "e4m3", "e5m2"])
        while True:
            T, D = _log(rng, 1, 16384), rng.choice([_log(rng, 64, 16384), 128 * _log(rng, 1, 128)])
            if T * D <= 8192 * 4096:
                break
        return {"op": op, "T": T, "D": D, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "wdtype": rng.choice(["bf16", "f32"]) if out == "same" else "f32", "residual": rng.random() < 0.7,
                "out": out, "train": out == "same" and rng.random() < 0.5}
    if op == "linear":
        mode = rng.choice(["forward", "forward", "products", "act"])
        while True:
            M = _log(rng, 1, 8192)
            N = rng.choice([_log(rng, 128, 16384), 128 * rng.randint(1, 128)])
            K = rng.choice([_log(rng, 128, 8192), 128 * rng.randint(1, 64), 128 * rng.randint(1, 64)])
            if M * N * K * (2 if mode == "products" else 1) <= 8192 * 16384 * 4096:
                break
        if mode == "act":
            return {"op": op, "mode": mode, "M": M, "N": N, "act": rng.choice(_ACTS)}
        if mode == "products":
            return {"op": op, "mode": mode, "M": M, "N": N, "K": K, "act": rng.choice(_ACTS), "out": rng.choice(["bf16", "f32"])}
        return {"op": op, "mode": mode, "M": M, "N": N, "K": K, "act": rng.choice(_ACTS), "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.4, "pre": rng.random() < 0.4, "out": rng.choice(["bf16", "bf16", "f32"])}
    while True:
        matrices, rows, cols = _log(rng, 1, 256), _log(rng, 8, 16384), rng.choice([_log(rng, 8, 8192), 64 * rng.randint(1, 64)])
        if matrices * rows * cols <= 2 * 16384 * 4096:
            break
    dtype = rng.choice(["f32", "bf16"])
    return {"op": op, "matrices": matrices, "rows": rows, "cols": cols, "vectors": rng.randint(0, 64),
            "odd": rng.randint(0, 8), "dtype": dtype, "out": rng.choice([dtype, "f32"]), "ratio": rng.choice([0.1, 0.5, 2.0])}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _activations(g, T, D, dtype):
    """Rows and columns of very different sizes, as a residual stream's are."""
    return (torch.randn(T, D, generator=g, device="cuda") * torch.exp(_normal(g, T, 1, std=0.5)) *
            torch.exp(_normal(g, 1, D, std=0.5))).to(dtype)


def _border_rows(case, st):
    """Rows in which a block's largest magnitude lies so near a scale's border that the last bits of
    a 32-bit result decide between two scales."""
    h = st["X"].double() + (st["residual"].double() if case["residual"] else 0.0)
    y = (h * torch.rsqrt((h * h).mean(1, keepdim=True) + _EPS) * st["w"].double()).abs()
    peak = torch.nn.functional.pad(y, (0, _up(case["D"], 128) - case["D"])).view(case["T"], -1, 128).amax(2)
    mant = torch.frexp(peak)[0]     # the border is at 0.875
    return ((mant - 0.875).abs() < 1e-5).any(1)


def _clip_shapes(case):
    return ([(case["rows"], case["cols"])] * case["matrices"] + [(case["cols"],)] * case["vectors"] +
            [(2 * i + 1, 37) for i in range(case["odd"])])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "norm":
        T, D, dt = case["T"], case["D"], _DT[case["dtype"]]
        st["X"] = _activations(g, T, D, dt)
        st["residual"] = _activations(g, T, D, dt) if case["residual"] else None
        st["w"] = (1 + _normal(g, D, std=0.2)).to(_DT[case["wdtype"]])
        if case["out"] != "same":
            for _ in range(8):
                close = _border_rows(case, st)
                n = int(close.sum())
                if n == 0:
                    break
                st["X"][close] = _activations(g, n, D, dt)
        if case["train"]:
            st["dY"] = _normal(g, T, D, std=0.01, dtype=dt)
            st["dH"] = _normal(g, T, D, std=0.01, dtype=dt) if case["residual"] else None
        return st
    if case["op"] == "linear":
        M, N, bf = case["M"], case["N"], torch.bfloat16
        if case["mode"] == "act":
            st["dY"], st["pre"] = _normal(g, M, N, std=0.01, dtype=bf), _normal(g, M, N, std=1.5, dtype=bf)
            return st
        K = case["K"]
        st["W"] = _normal(g, N, K, std=K ** -0.5, dtype=bf)
        st["X"] = _normal(g, M, K, dtype=bf)
        if case["mode"] == "forward":
            st["bias"] = _normal(g, N, std=0.1, dtype=bf) if case["bias"] else None
            st["residual"] = _normal(g, M, N, dtype=bf) if case["residual"] else None
        else:
            st["dZ"] = _normal(g, M, N, std=0.01, dtype=bf)
            # X = act(pre): what the activation before this product saw
            st["pre"] = _normal(g, M, K, std=1.5, dtype=bf) if case["act"] != "none" else None
        return st
    dt = _DT[case["dtype"]]
    st["grads"] = [_normal(g, *shape, std=0.01 * (1 + i % 3), dtype=dt) for i, shape in enumerate(_clip_shapes(case))]
    # the scaled gradients go to one buffer, as an optimizer keeps them: each tensor's part starts at a
    # multiple of 64 elements
    starts, end = [], 0
    for t in st["grads"]:
        starts.append(end)
        end += _up(t.numel(), 64)
    st["flat"] = torch.zeros(end, dtype=_DT[case["out"]], device="cuda")
    st["out"] = [st["flat"][a:a + t.numel()].view(t.shape) for a, t in zip(starts, st["grads"])]
    st["max_norm"] = case["ratio"] * 0.02 * math.sqrt(sum(t.numel() for t in st["grads"]))
    return st


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return (_OWN if own else _PLAIN)[case["op"]](case, state)


def _blocks_plain(y, fmt):
    """y [T, D] in 32 bits -> Q [T, Dp] in 8 bits and the power-of-two scales S [Dp / 128, T]."""
    T, D = y.shape
    x = torch.nn.functional.pad(y, (0, _up(D, 128) - D)).view(T, -1, 128)
    amax = x.abs().amax(2)
    mant, expo = torch.frexp(amax)
    # amax = mant 2^expo with mant in [0.5, 1), the format's largest value 0.875 * 2^top
    expo = (expo - (9 if fmt == "e4m3" else 16) + (mant > 0.875).int()).clamp(min=-126)
    s = torch.where(amax > 0, ((expo + 127) << 23).view(torch.float32), torch.ones_like(amax))
    return (x / s.unsqueeze(2)).to(_F8[fmt]).view(T, -1), s.t().contiguous()


def _norm_plain(case, st):
    dt = _DT[case["dtype"]]
    h = st["X"].float()
    if case["residual"]:
        h = h + st["residual"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + _EPS)
    y = h * rstd * st["w"].float()
    H = h.to(dt)
    out = [y.to(dt)] if case["out"] == "same" else [*_blocks_plain(y, case["out"])]
    out += [H, rstd.squeeze(1)]
    if case["train"]:
        xh = H.float() * rstd
        dy = st["dY"].float()
        gw = dy * st["w"].float()
        dx = rstd * (gw - xh * (gw * xh).mean(1, keepdim=True))
        if st["dH"] is not None:
            dx = dx + st["dH"].float()
        out += [dx.to(dt), (dy * xh).sum(0)]
    return out


def _norm_own(case, st):
    import sparse_matmul_ffns_amd as nm
    if case["out"] != "same":
        Q, S, H, rstd = nm.rms_norm_fp8(st["X"], st["w"], eps=_EPS, residual=st["residual"], fmt=_F8[case["out"]])
        return [Q, S, H, rstd]
    out = list(nm.rms_norm(st["X"], st["w"], eps=_EPS, residual=st["residual"]))
    if case["train"]:
        out += nm.rms_norm_bwd(st["dY"], out[1], st["w"], out[2], dH=st["dH"])
    return out


def _act_plain(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _dact_plain(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _linear_plain(case, st):
    bf = torch.bfloat16
    if case["mode"] == "act":
        dz = st["dY"].float() * _dact_plain(st["pre"].float(), case["act"])
        return [dz.to(bf), dz.sum(0)]
    if case["mode"] == "products":
        dz = st["dZ"].float()
        dx = torch.matmul(dz, st["W"].float())
        if st["pre"] is not None:
            dx = dx * _dact_plain(st["pre"].float(), case["act"])
        return [dx.to(_DT[case["out"]]), torch.matmul(dz.t(), st["X"].float())]
    z = torch.matmul(st["X"].float(), st["W"].float().t())
    if case["bias"]:
        z = z + st["bias"].float()
    y = _act_plain(z, case["act"])
    if case["residual"]:
        y = y + st["residual"].float()
    y = y.to(_DT[case["out"]])
    return [y, z.to(bf)] if case["pre"] else [y]


def _linear_own(case, st):
    import sparse_matmul_ffns_amd as nm
    if case["mode"] == "act":
        return list(nm.linear_bwd_act(st["dY"], st["pre"], act=case["act"]))
    if case["mode"] == "products":
        return [nm.linear_bwd_x(st["dZ"], st["W"], pre=st["pre"], act=case["act"], out_dtype=_DT[case["out"]]),
                nm.linear_bwd_w(st["dZ"], st["X"])]
    y = nm.linear_fwd(st["X"], st["W"], bias=st["bias"], act=case["act"], residual=st["residual"],
                      out_dtype=_DT[case["out"]], return_pre=case["pre"])
    return list(y) if case["pre"] else [y]


def _clip_plain(case, st):
    total = torch.stack([(t.float() * t.float()).sum(dtype=torch.float64) for t in st["grads"]]).sum()
    norm = torch.sqrt(total)
    factor = torch.where(norm > st["max_norm"], st["max_norm"] / norm, torch.ones_like(norm)).float()
    _ = [o.copy_(t.float() * factor) for t, o in zip(st["grads"], st["out"])]
    return [norm.float().view(1), st["flat"]]


def _clip_own(case, st):
    import sparse_matmul_ffns_amd as nm
    return [nm.grad_clip(st["grads"], st["max_norm"], out=st["out"]), st["flat"]]


_PLAIN = {"norm": _norm_plain, "linear": _linear_plain, "clip": _clip_plain}
_OWN = {"norm": _norm_own, "linear": _linear_own, "clip": _clip_own}


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    es = {"bf16": 2, "f32": 4}
    if case["op"] == "norm":
        T, D, e = case["T"], case["D"], es[case["dtype"]]
        n = T * D
        # in: the rows and what is added to them; out: the sum (the input itself where nothing is added)
        b = n * e * (3 if case["residual"] else 1) + D * es[case["wdtype"]] + T * 4
        b += n * e if case["out"] == "same" else n + T * _up(D, 128) // 32
        f = 5 * n
        if case["train"]:
            b += n * e * (4 if case["residual"] else 3) + D * 4
            f += 9 * n
        return {"bytes": b, "flops": f}
    if case["op"] == "linear":
        M, N = case["M"], case["N"]
        if case["mode"] == "act":
            return {"bytes": 3 * 2 * M * N + 4 * N, "flops": 10 * M * N}
        K = case["K"]
        if case["mode"] == "products":
            b = 2 * (M * N + N * K + M * K) + (2 * M * K if case["act"] != "none" else 0)
            return {"bytes": b + M * K * es[case["out"]] + 4 * N * K, "flops": 4 * M * N * K}
        b = 2 * (M * K + N * K) + M * N * es[case["out"]]
        b += 2 * N * case["bias"] + 2 * M * N * case["residual"] + 2 * M * N * case["pre"]
        return {"bytes": b, "flops": 2 * M * N * K}
    n = sum(math.prod(shape) for shape in _clip_shapes(case))
    return {"bytes": n * (es[case["dtype"]] + es[case["out"]]), "flops": 3 * n}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _power64(e):
    return torch.ldexp(torch.ones((), dtype=torch.float64, device=e.device), e)


def _round8_64(v, fmt):
    """v in 64 bits, within the format's range, to the nearest 8-bit value, ties to even."""
    digits, lowest = (3, -6) if fmt == "e4m3" else (2, -14)
    step = _power64((torch.frexp(v)[1] - 1).clamp(min=lowest) - digits)
    return torch.round(v / step) * step


def _norm_exact(case, st):
    dt, T, D = _DT[case["dtype"]], case["T"], case["D"]
    h = st["X"].double()
    if case["residual"]:
        h += st["residual"].double()
    r = (h.square().sum(1) / D + _EPS).pow(-0.5)
    w = st["w"].double()
    y = torch.einsum("td,t,d->td", h, r, w)
    if case["out"] == "same":
        out = [y]
    else:
        Dp = _up(D, 128)
        full = torch.zeros(T, Dp, dtype=torch.float64, device=y.device)
        full[:, :D] = y
        full = full.view(T, Dp // 128, 128)
        peak = full.abs().max(2)[0]
        power = torch.log2(peak / _TOP[case["out"]]).ceil().clamp(min=-126)
        scale = torch.where(peak > 0, torch.exp2(power), torch.ones_like(peak))
        scale = torch.where(scale * _TOP[case["out"]] < peak, 2 * scale, scale)
        out = [_round8_64(full / scale.unsqueeze(2), case["out"]).view(T, Dp), scale.t().contiguous()]
    out += [h, r]
    if case["train"]:
        # the gradient is taken at the stored sum
        hs = h.to(dt).double()
        dy = st["dY"].double()
        v = dy * w
        inner = (v * hs).sum(1) * r.pow(3) / D
        dx = v * r.unsqueeze(1) - hs * inner.unsqueeze(1)
        if st["dH"] is not None:
            dx += st["dH"].double()
        out += [dx, torch.matmul(r.unsqueeze(0), dy * hs).squeeze(0)]
    return out


def _exact_act(z, act):
    """The activation and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        on = z.gt(0).double()
        return z * on, on
    c, cube = (math.sqrt(8 / math.pi), 0.044715) if act == "gelu_tanh" else (1.0, 0.0)
    s = torch.sigmoid(c * z * (1 + cube * z.square()))
    return z * s, s + z * s * (1 - s) * c * (1 + 3 * cube * z.square())


def _linear_exact(case, st):
    if case["mode"] == "act":
        dz = st["dY"].double() * _exact_act(st["pre"].double(), case["act"])[1]
        return [dz, dz.sum(0)]
    x, w = st["X"].double(), st["W"].double()
    if case["mode"] == "products":
        dz = st["dZ"].double()
        dx = dz @ w
        if st["pre"] is not None:
            dx *= _exact_act(st["pre"].double(), case["act"])[1]
        return [dx, dz.t() @ x]
    z = x @ w.t()
    if st["bias"] is not None:
        z += st["bias"].double()
    y = _exact_act(z, case["act"])[0]
    if st["residual"] is not None:
        y = y + st["residual"].double()
    return [y, z] if case["pre"] else [y]


def _clip_exact(case, st):
    norm = math.sqrt(math.fsum(float(t.double().square().sum()) for t in st["grads"]))
    factor = min(1.0, st["max_norm"] / norm) if norm else 1.0
    gaps = [t.new_zeros(-t.numel() % 64, dtype=torch.float64) for t in st["grads"]]
    parts = [p for t, gap in zip(st["grads"], gaps) for p in (t.double().reshape(-1) * factor, gap)]
    return [torch.tensor([norm], dtype=torch.float64), torch.cat(parts)]


_EXACT = {"norm": _norm_exact, "linear": _linear_exact, "clip": _clip_exact}
