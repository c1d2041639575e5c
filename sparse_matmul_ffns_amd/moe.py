"""A mixture-of-experts FFN in 8-bit floating point over the library's calls.

"To 2:4 Sparsity and Beyond" (abstract) states that its FFN method is orthogonal to quantisation and
applies to mixture-of-experts; this module is the mixture-of-experts FFN itself, each expert the up-
projection, ReLU and down-projection of the framework's FFN:

    y[t] = sum_j w[t, j] W_down[e_j] relu(W_up[e_j] x[t]),   (e, w) = moe_route(logits)

It only sequences the library's calls (and torch allocations); nothing here computes on tensors.

    python -c "from sparse_matmul_ffns_amd import moe; moe.main()"

runs one forward and backward pass of a layer of 64 experts and prints its time.
"""

from __future__ import annotations

import torch

from . import nmsparse as _nm


def _version(t: torch.Tensor):
    """torch's count of the in-place changes of t (tensors made in inference mode have none)."""
    return None if t.is_inference() else t._version


class ExpertFFN:
    """The experts' weights W_up [E, F, D] and W_down [E, D, F] (bf16 or fp32, device) held in 8 bits,
    and the calls of a forward and a backward pass.

    `train` keeps the weights' transposed bytes too, orders the rows by expert in runs of 128 (what the
    weight gradients' blocks need) and saves what backward() reads; without it a pass keeps nothing.
    The layer keeps the last pass only, and with it x and logits themselves, not copies.  Passes that wait
    for their gradients together (micro-batches, threads) are kept by the caller: forward(...,
    return_saved=True) and backward(dy, saved).
    Routing options as for moe_route; activations and weights are e4m3, gradients `grad_fmt`."""

    def __init__(self, W_up: torch.Tensor, W_down: torch.Tensor, k: int, score: str = "softmax", bias=None,
                 groups: int = 1, topk_groups: int = 1, group_top: int = 2, renorm: bool = True, scale: float = 1.0,
                 train: bool = False, grad_fmt: torch.dtype = torch.float8_e5m2):
        if W_up.dim() != 3:
            raise ValueError("W_up must be [E, F, D]")
        self.E, self.F, self.D = W_up.shape
        self.k, self.train, self.grad_fmt = k, train, grad_fmt
        self.choice = dict(bias=bias, groups=groups, topk_groups=topk_groups, group_top=group_top)
        self.score = dict(score=score, renorm=renorm, scale=scale)
        self.saved = None
        self.used = self.replaced = False   # the saved pass has had a backward pass; it replaced one that had none
        self.generation = 0                 # of the weights
        self.set_weights(W_up, W_down)

    def set_weights(self, W_up: torch.Tensor, W_down: torch.Tensor) -> None:
        """Quantise the weights (again, after an optimizer step); their shapes stay those of the layer."""
        E, F, D = self.E, self.F, self.D
        if tuple(W_up.shape) != (E, F, D) or tuple(W_down.shape) != (E, D, F):
            raise ValueError(f"W_up must be [E, F, D] = {[E, F, D]} and W_down [E, D, F]")
        self.generation += 1
        self.up = _nm.fp8_quantize_weight(W_up, transposed=self.train)
        self.down = _nm.fp8_quantize_weight(W_down, transposed=self.train)

    def forward(self, x: torch.Tensor, logits: torch.Tensor, return_saved: bool = False):
        """y [T, D] of tokens x [T, D] (bf16) and router logits [T, E]; with `return_saved` (y, what
        backward() reads), and the layer itself keeps nothing of the pass."""
        if return_saved and not self.train:
            raise ValueError("return_saved needs a layer with train=True")
        # the products pad D to 128 and the plan drops choices of no expert: neither would notice
        if x.dim() != 2 or x.shape[1] != self.D:
            raise ValueError(f"x must be [T, {self.D}]")
        if logits.shape != (x.shape[0], self.E):
            raise ValueError(f"logits must be [T, {self.E}] with x's number of tokens")
        ids, w = _nm.moe_route(logits, self.k, **self.choice, **self.score)
        offsets, _, src, pos = _nm.moe_plan(ids, self.E, align=128 if self.train else 1)
        q, s = _nm.fp8_quantize(x, src=src, div=self.k)
        h = _nm.fp8_gemm_nt_grouped(q, s, self.up[0], self.up[1], offsets, out_dtype=x.dtype)
        q, s = _nm.fp8_quantize(h, gate=h)
        o = _nm.fp8_gemm_nt_grouped(q, s, self.down[0], self.down[1], offsets, out_dtype=x.dtype)
        y = _nm.moe_combine(o, pos, w)
        if not self.train:
            return y
        saved = (x, logits, ids, w, offsets, src, pos, h, o, self.generation, _version(x), _version(logits))
        if return_saved:
            return y, saved
        self.replaced = self.saved is not None and not self.used
        self.saved, self.used = saved, False
        return y

    def backward(self, dy: torch.Tensor, saved=None):
        """Gradients of the last forward pass, or of the one that returned `saved`: (dx [T, D], dlogits
        [T, E], dW_up [E, F, D] and dW_down [E, D, F] in fp32).

        Refused (RuntimeError): a second backward() of a pass that took the place of one without
        a backward pass, as two forwards and then two backwards make it; x, logits (by torch's calls or this library's) or
        the weights changed since the pass."""
        if saved is None:
            saved = self.saved
            if saved is None:
                raise RuntimeError("backward() needs a forward pass with train=True")
            if self.used and self.replaced:
                raise RuntimeError("the layer keeps the last pass only, and an earlier one had no backward(): keep the "
                                   "passes with forward(..., return_saved=True) and give each to backward(dy, saved)")
        x, logits, ids, w, offsets, src, pos, h, o, generation, *versions = saved
        if generation != self.generation:
            raise RuntimeError("the weights have been set since this forward pass")
        if versions != [_version(x), _version(logits)]:
            raise RuntimeError("x or logits has been changed in place since this forward pass")
        g = self.grad_fmt
        do, dw = _nm.moe_combine_bwd(dy, o, src, pos, w)
        dlogits = _nm.moe_route_bwd(logits, ids, w, dw, **self.score)
        q, s = _nm.fp8_quantize(do, g)
        dh = _nm.fp8_gemm_nt_grouped(q, s, self.down[2], self.down[3], offsets, out_dtype=x.dtype)
        dW_down = _nm.fp8_gemm_nt_grouped_k(*_nm.fp8_quantize_t(do, g), *_nm.fp8_quantize_t(h, gate=h), offsets)
        q, s = _nm.fp8_quantize(dh, g, gate=h)
        dx = _nm.moe_combine(_nm.fp8_gemm_nt_grouped(q, s, self.up[2], self.up[3], offsets, out_dtype=x.dtype), pos)
        dW_up = _nm.fp8_gemm_nt_grouped_k(*_nm.fp8_quantize_t(dh, g, gate=h),
                                          *_nm.fp8_quantize_t(x, src=src, div=self.k), offsets)
        if saved is self.saved:
            self.used = True
        return dx, dlogits, dW_up, dW_down


def main(tokens: int = 4096) -> None:
    E, D, F, k = 64, 2048, 1024, 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *shape, std=1.0: (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()
    layer = ExpertFFN(rand(E, F, D, std=0.02), rand(E, D, F, std=0.02), k, train=True)
    x, dy, logits = rand(tokens, D), rand(tokens, D), rand(tokens, E).float()
    times = []
    for _ in range(5):
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        marks[0].record()
        y = layer.forward(x, logits)
        marks[1].record()
        grads = layer.backward(dy)
        marks[2].record()
        torch.cuda.synchronize()
        times.append((marks[0].elapsed_time(marks[1]), marks[1].elapsed_time(marks[2])))
    fwd, bwd = (min(t) for t in zip(*times))
    assert all(bool(torch.isfinite(t).all()) for t in (y, *grads))
    flops = 4 * tokens * k * D * F
    print(f"{tokens} tokens, {k} of {E} experts, {D} x {F}: forward {fwd:.3f} ms ({flops / fwd / 1e9:.0f} TFLOP/s), "
          f"backward {bwd:.3f} ms ({2 * flops / bwd / 1e9:.0f} TFLOP/s)")

