"""Every call of the binding counts the change of the outputs that it was given, as torch counts its own in-place changes (CPU: the
library is replaced by one that returns a status and writes nothing)."""

import inspect

import pytest
import torch

from sparse_matmul_ffns_amd import dense, moe, nmsparse as nm


class Library:
    status = 0

    def __getattr__(self, name):
        return lambda *args: self.status


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(nm, "lib", lambda: L)
    monkeypatch.setattr(nm, "_dev", lambda *ts: None)
    monkeypatch.setattr(nm, "_here", lambda *ts: None)
    monkeypatch.setattr(nm, "_here_all", lambda ts: None)
    monkeypatch.setattr(nm, "_stream", lambda: None)
    monkeypatch.setattr(nm, "sizes", lambda R, K, N=2, M=4, V=0: (R * K // 2, R * K // 8, 4))
    for name in ("_plan_work_bytes", "_norm_work_bytes", "_linear_work_bytes", "_act_work_bytes", "general_work_bytes",
                 "venom_tn_work_bytes"):
        monkeypatch.setattr(nm, name, lambda *args: 0)

    def refuse(status, call):
        if status:
            raise RuntimeError(call)
    monkeypatch.setattr(nm, "_check", refuse)
    return L


def b(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def f(*shape):
    return torch.zeros(*shape)


def u(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def q(*shape):
    return u(*shape).view(torch.float8_e4m3fn)


# a call's inputs, and its outputs
CALLS = {
    "nm_prune": (dict(A=b(8, 16)), dict(mask=u(8, 16))),
    "nm_compress": (dict(A=b(8, 16), mask=u(8, 16)), dict(bad_groups=i(1), values=b(8, 8), meta=u(8, 2))),
    "nm_prune_compress": (dict(A=b(8, 16)), dict(mask=u(8, 16), values=b(8, 8), meta=u(8, 2))),
    "nm_prune_compress_transpose": (dict(A=b(8, 16), B=b(4, 8)), dict(mask=u(8, 16), values=b(8, 8), meta=u(8, 2), Bt=b(8, 4))),
    "nm_decompress": (dict(values=b(8, 8), meta=u(8, 2), K=16), dict(out=b(8, 16))),
    "spmm_nm": (dict(values=b(8, 8), meta=u(8, 2), K=16, B=b(16, 4)), dict(out=f(8, 4))),
    "spmm_nm_t": (dict(values=b(8, 8), meta=u(8, 2), K=16, Bt=b(4, 16)), dict(out=f(8, 4))),
    "spmm_nm_t bf16": (dict(values=b(8, 8), meta=u(8, 2), K=16, Bt=b(4, 16)), dict(out=b(8, 4))),
    "spmm_nm_t_lowrank": (dict(values=b(8, 8), meta=u(8, 2), K=16, Bt=b(4, 16), U=b(8, 2), Vt=b(2, 16)), dict(out=f(8, 4), Tt=f(4, 2))),
    "spmm_nm_t_relu_venom": (dict(values=b(8, 8), meta=u(8, 2), K=16, Bt=b(4, 16), V=4), dict(h_values=b(4, 4), h_meta=u(4, 1), h_colsel=u(1, 1, 4))),
    "spmm_nm_general": (dict(values=b(8, 8), meta=u(8, 2), K=16, N=2, M=4, Bt=b(4, 16)), dict(out=f(8, 4))),
    "spmm_nm_general_noalloc": (dict(values=b(8, 8), meta=u(8, 2), K=16, N=2, M=4, Bt=b(4, 16)), dict(out=f(8, 4))),
    "sddmm_venom": (dict(dY=b(4, 6), W_down=b(16, 6), h_values=b(4, 4), h_meta=u(4, 4), h_colsel=u(4), V=4), dict(out=f(4, 4), dYt=b(6, 4))),
    "spmm_venom_tn": (dict(h_values=b(4, 4), h_meta=u(4, 4), h_colsel=u(4), F=16, V=4, M=8, dYt=b(6, 4)), dict(out=f(16, 6))),
    "transpose": (dict(X=b(4, 6)), dict(out=b(6, 4))),
    "prune_act_venom": (dict(Z=b(8, 16), V=4), dict(values=b(8, 8), meta=u(8, 2), colsel=u(2, 2, 4), mask=u(8, 16))),
    "spmm_venom": (dict(values=b(8, 8), meta=u(8, 2), colsel=u(4), K=16, V=4, M=8, B=b(16, 4)), dict(out=f(8, 4))),
    "nm_reprune_t": (dict(values=b(8, 8), meta=u(8, 2), R=8, K=16), dict(values_t=b(16, 4), meta_t=u(16, 1))),
    "nm_reprune_t_transpose": (dict(values=b(8, 8), meta=u(8, 2), R=8, K=16, X=b(4, 6)), dict(values_t=b(16, 4), meta_t=u(16, 1), Xt=b(6, 4))),
    "mfma_rate_probe": (dict(kind=0, iters=1), dict(sink=f(512 * 256))),
    "nm_to_panels": (dict(values=b(8, 8), meta=u(8, 2), R=8, K=16), dict(values_p=b(64), meta_p=u(16))),
    "nm_reprune_t_transpose_panels": (dict(values=b(8, 8), meta=u(8, 2), R=8, K=16, X=b(4, 6)), dict(values_t=b(64), meta_t=u(16), Xt=b(6, 4))),
    "spmm_nm_t_panels": (dict(values=b(64), meta=u(16), R=8, K=16, Bt=b(4, 16)), dict(out=f(8, 4))),
    "sddmm_nm": (dict(D=b(8, 4), X=b(16, 4), meta=u(8, 2)), dict(out=f(8, 8))),
    "sddmm_nm dt": (dict(D=b(8, 4), X=b(16, 4), meta=u(8, 2)), dict(out=f(8, 8), Dt=b(4, 8))),
    "moe_route": (dict(logits=b(4, 8), k=2), dict(ids=i(4, 2), weights=f(4, 2))),
    "moe_route_bwd": (dict(logits=b(4, 8), ids=i(4, 2), weights=f(4, 2), dweights=f(4, 2)), dict(dlogits=b(4, 8))),
    "moe_plan": (dict(ids=i(4, 2), E=8), dict(offsets=i(9), counts=i(8), src=i(8), pos=i(4, 2))),
    "fp8_quantize": (dict(X=b(4, 128)), dict(Q=q(4, 128), S=f(1, 4))),
    "fp8_quantize_t": (dict(X=b(128, 4)), dict(Q=q(4, 128), S=f(1, 4))),
    "fp8_gemm_nt": (dict(A=q(4, 128), sa=f(1, 4), B=q(128, 128), sb=f(1, 1)), dict(out=b(4, 128))),
    "fp8_gemm_nt_grouped": (dict(A=q(4, 128), sa=f(1, 4), B=q(2, 128, 128), sb=f(2, 1, 1), offsets=i(3)), dict(out=b(4, 128))),
    "fp8_gemm_nt_grouped_k": (dict(A=q(4, 128), sa=f(1, 4), B=q(6, 128), sb=f(1, 6), offsets=i(3)), dict(out=f(2, 4, 6))),
    "moe_combine": (dict(O=b(8, 16), pos=i(4, 2)), dict(out=b(4, 16))),
    "moe_combine_bwd": (dict(dY=b(4, 16), O=b(8, 16), src=i(8), pos=i(4, 2), weights=f(4, 2)), dict(dO=b(8, 16), dweights=f(4, 2))),
    "rms_norm": (dict(X=b(4, 16), w=f(16), residual=b(4, 16)), dict(H=b(4, 16), Y=b(4, 16), rstd=f(4))),
    "rms_norm_fp8": (dict(X=b(4, 16), w=f(16), residual=b(4, 16)), dict(H=b(4, 16), Q=q(4, 128), S=f(1, 4), Y=b(4, 16), rstd=f(4))),
    "rms_norm_bwd": (dict(dY=b(4, 16), H=b(4, 16), w=f(16), rstd=f(4), dH=b(4, 16)), dict(dX=b(4, 16), dw=f(16))),
    "linear_fwd": (dict(X=b(4, 16), W=b(8, 16), bias=b(8), residual=b(4, 8)), dict(out=b(4, 8), pre=b(4, 8))),
    "linear_bwd_act": (dict(dY=b(4, 8), pre=b(4, 8), act="silu"), dict(dZ=b(4, 8), db=f(8))),
    "linear_bwd_x": (dict(dZ=b(4, 8), W=b(8, 16), pre=b(4, 16), act="relu"), dict(out=b(4, 16))),
    "linear_bwd_w": (dict(dZ=b(4, 8), X=b(4, 16)), dict(out=f(8, 16))),
    "grad_norm": (dict(grads=[f(3), b(4)]), dict(norm=f(1))),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_given_outputs(library, name):
    call, (inputs, outputs) = getattr(nm, name.split()[0]), CALLS[name]
    read = [t for t in inputs.values() if torch.is_tensor(t)]
    seen = [t._version for t in read]
    before = {k: t._version for k, t in outputs.items()}
    library.status = 2
    with pytest.raises(RuntimeError):
        call(**inputs, **outputs)
    assert {k: t._version for k, t in outputs.items()} == before      # nothing was written
    library.status = 0
    call(**inputs, **outputs)
    assert {k: t._version for k, t in outputs.items()} == {k: v + 1 for k, v in before.items()}
    assert [t._version for t in read] == seen
    needed = [k for k in outputs if inspect.signature(call).parameters[k].default is inspect.Parameter.empty]
    if not needed:
        call(**inputs)


def test_every_call_with_outputs_is_here():
    """The binding's public functions that reach a kernel."""
    names = {n for n, v in vars(nm).items() if inspect.isfunction(v) and not n.startswith("_") and "_stream()" in inspect.getsource(v)}
    allocates_all = {"fp8_quantize_weight"}
    assert names - allocates_all - {"grad_clip"} == {n.split()[0] for n in CALLS}


def test_clipping(library):
    g, o, norm = [f(3), b(4)], [f(3), f(4)], f(1)
    for t in g + o:
        assert t._version == 0
    nm.grad_clip(g, 1.0)
    assert [t._version for t in g] == [1, 1]
    nm.grad_clip(g, 1.0, norm=norm, out=o)
    assert [t._version for t in g] == [1, 1] and [t._version for t in o] == [1, 1] and norm._version == 0


def test_views_and_inference(library):
    x = b(8, 32)
    nm.rms_norm(b(4, 16), f(16), residual=x[:4, :16], H=x[:4, :16])
    assert x._version == 1
    with torch.inference_mode():
        t = b(4, 16)
        nm.rms_norm(t, f(16), Y=t)                    # has no count


def test_layers_see_the_library_write(library):
    x, dy = b(4, 16), b(4, 16)
    layer = dense.DenseFFN(f(16), b(24, 16), b(16, 24), train=True)
    layer.forward(x)
    layer.backward(dy)
    nm.rms_norm(b(4, 16), f(16), residual=x, H=x)
    with pytest.raises(RuntimeError):
        layer.backward(dy)
    experts = moe.ExpertFFN(b(2, 24, 16), b(2, 16, 24), k=2, train=True)
    experts.forward(x, b(4, 2))
    nm.linear_fwd(b(4, 8), b(16, 8), residual=x, out=x)
    with pytest.raises(RuntimeError):
        experts.backward(dy)
