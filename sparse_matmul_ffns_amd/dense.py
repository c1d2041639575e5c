"""A dense FFN block over the library's calls: the residual's addition, the norm, both products and their gradients.

"To 2:4 Sparsity and Beyond" (abstract) trains with sparse steps and switches to "regular dense training steps
towards the end"; this module is the block of those steps, in bf16 with fp32 sums:

    h = x + residual;  y = h + W_down act(W_up norm(h) + b_up) + b_down

It only sequences the library's calls (and torch allocations); nothing here computes on tensors.

    python -c "from sparse_matmul_ffns_amd import dense; dense.main()"

runs training steps of a block of d_model 4096 and d_ff 16384 over 8192 tokens, gradients clipped, and prints their time.
"""

from __future__ import annotations

import torch

from . import nmsparse as _nm
from .moe import _version


class DenseFFN:
    """The block's norm weight [D] and weights W_up [F, D] and W_down [D, F] with biases [F] and [D] (None: none), bf16 (the
    norm's and the biases also fp32), held by reference.

    With `train` a pass saves what backward() reads; the layer keeps the last pass only, and with it x and residual
    themselves, not copies.  Passes that wait for their gradients together (micro-batches, threads) are kept by the caller:
    forward(..., return_saved=True) and backward(dy, saved)."""

    def __init__(self, w_norm: torch.Tensor, W_up: torch.Tensor, W_down: torch.Tensor, b_up=None, b_down=None,
                 act: str = "gelu_tanh", eps: float = 1e-5, train: bool = False):
        if W_up.dim() != 2 or W_down.shape != (W_up.shape[1], W_up.shape[0]):
            raise ValueError("W_up must be [F, D] and W_down [D, F]")
        self.F, self.D = W_up.shape
        for name, v, n in (("w_norm", w_norm, self.D), ("b_up", b_up, self.F), ("b_down", b_down, self.D)):
            if v is not None and v.shape != (n,):
                raise ValueError(f"{name} must be [{n}]")
        _nm._act(act)
        self.w_norm, self.W_up, self.W_down, self.b_up, self.b_down = w_norm, W_up, W_down, b_up, b_down
        self.act, self.eps, self.train = act, eps, train
        self.saved = None
        self.used = self.replaced = False   # the saved pass has had a backward pass; it replaced one that had none

    def parameters(self):
        """The block's parameters, in the order of backward()'s gradients."""
        return [p for p in (self.w_norm, self.W_up, self.W_down, self.b_up, self.b_down) if p is not None]

    def forward(self, x: torch.Tensor, residual=None, return_saved: bool = False):
        """y [T, D] of x [T, D] (bf16); with `return_saved` (y, what backward() reads), and the layer itself keeps
        nothing of the pass."""
        if return_saved and not self.train:
            raise ValueError("return_saved needs a layer with train=True")
        if x.dim() != 2 or x.shape[1] != self.D:
            raise ValueError(f"x must be [T, {self.D}]")
        n, h, rstd = _nm.rms_norm(x, self.w_norm, eps=self.eps, residual=residual)
        # ReLU's derivative follows from the activations themselves
        keep = self.train and self.act not in ("none", "relu")
        a = _nm.linear_fwd(n, self.W_up, bias=self.b_up, act=self.act, return_pre=keep)
        a, pre = a if keep else (a, a)
        y = _nm.linear_fwd(a, self.W_down, bias=self.b_down, residual=h)
        if not self.train:
            return y
        read = [x] if residual is None else []                  # h is x itself then
        read += self.parameters()
        saved = (h, rstd, n, pre, a, read, [_version(t) for t in read])
        if return_saved:
            return y, saved
        self.replaced = self.saved is not None and not self.used
        self.saved, self.used = saved, False
        return y

    def backward(self, dy: torch.Tensor, saved=None):
        """The gradients of the last forward pass, or of the one that returned `saved`: dx [T, D] (of x and of residual), and
        those of parameters(), in their order and fp32.  The gradients between the products are bf16: b_up's is the fp32 sum of what
        W_up's is a product of, the rounded gradient behind the activation.

        Refused (RuntimeError): a second backward() of a pass that took the place of one without a backward pass; x or the
        parameters changed in place since the pass, by torch's calls or by this library's (a tensor's version counts both)."""
        if saved is None:
            saved = self.saved
            if saved is None:
                raise RuntimeError("backward() needs a forward pass with train=True")
            if self.used and self.replaced:
                raise RuntimeError("the layer keeps the last pass only, and an earlier one had no backward(): keep the "
                                   "passes with forward(..., return_saved=True) and give each to backward(dy, saved)")
        h, rstd, n, pre, a, read, versions = saved
        if versions != [_version(t) for t in read]:
            raise RuntimeError("x or a parameter has been changed in place since this forward pass")
        if dy.shape != h.shape:
            raise ValueError(f"dy must be {list(h.shape)}")
        dW_down = _nm.linear_bwd_w(dy, a)
        dz = _nm.linear_bwd_x(dy, self.W_down, pre=None if self.act == "none" else pre, act=self.act)
        dW_up = _nm.linear_bwd_w(dz, n)
        dx, dw = _nm.rms_norm_bwd(_nm.linear_bwd_x(dz, self.W_up), h, self.w_norm, rstd, dH=dy)
        grads = [dw, dW_up, dW_down]
        grads += [] if self.b_up is None else [_nm.linear_bwd_act(dz)[1]]
        grads += [] if self.b_down is None else [_nm.linear_bwd_act(dy)[1]]
        if saved is self.saved:
            self.used = True
        return dx, grads


def main(tokens: int = 8192) -> None:
    D, F = 4096, 16384
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *shape, std=1.0: (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()
    layer = DenseFFN(1 + rand(D, std=0.1), rand(F, D, std=D ** -0.5), rand(D, F, std=F ** -0.5), rand(F, std=0.1),
                     rand(D, std=0.1), train=True)
    x, residual, dy = rand(tokens, D), rand(tokens, D), rand(tokens, D)
    times = []
    for _ in range(5):
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
        marks[0].record()
        y = layer.forward(x, residual)
        marks[1].record()
        dx, grads = layer.backward(dy)
        marks[2].record()
        norm = _nm.grad_clip(grads, 1.0)
        marks[3].record()
        torch.cuda.synchronize()
        times.append([a.elapsed_time(b) for a, b in zip(marks, marks[1:])])
    fwd, bwd, clip = (min(t) for t in zip(*times))
    assert all(bool(torch.isfinite(t).all()) for t in (y, dx, norm, *grads))
    flops = 4 * tokens * D * F
    print(f"{tokens} tokens, {D} x {F}: forward {fwd:.3f} ms ({flops / fwd / 1e9:.0f} TFLOP/s), backward {bwd:.3f} ms "
          f"({2 * flops / bwd / 1e9:.0f} TFLOP/s), clipping {clip:.3f} ms")
