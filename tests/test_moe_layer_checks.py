"""What ExpertFFN refuses (CPU): the library's calls are replaced by a recorder, so that a check which
comes after a call shows too."""

import pytest
import torch

from sparse_matmul_ffns_amd import moe

E, D, F, K = 6, 200, 136, 3


class Called(Exception):
    pass


class Calls:
    """Stands for the binding: the weights' quantisation works, any other call is recorded by raising."""

    def __getattr__(self, name):
        def call(*args, **kw):
            raise Called(name)
        return call

    def fp8_quantize_weight(self, W, transposed=False):
        return ("q", "s", "qt", "st")[:4 if transposed else 2]


@pytest.fixture(params=[False, True])
def layer(request, monkeypatch):
    monkeypatch.setattr(moe, "_nm", Calls())
    return moe.ExpertFFN(torch.zeros(E, F, D), torch.zeros(E, D, F), K, train=request.param)


def test_forward_refuses_other_shapes(layer):
    with pytest.raises(Called):
        layer.forward(torch.zeros(5, D), torch.zeros(5, E))
    for x, logits in ((torch.zeros(5, 250), torch.zeros(5, E)),          # the padding to 128 would hide both
                      (torch.zeros(5, 199), torch.zeros(5, E)),
                      (torch.zeros(5, D), torch.zeros(5, E + 1)),        # choices of no expert
                      (torch.zeros(5, D), torch.zeros(5, E - 1)),
                      (torch.zeros(5, D), torch.zeros(6, E)),            # tokens without a row
                      (torch.zeros(5, D), torch.zeros(4, E)),
                      (torch.zeros(1, 5, D), torch.zeros(5, E)), (torch.zeros(5, D), torch.zeros(5 * E))):
        with pytest.raises(ValueError):
            layer.forward(x, logits)


def test_weights_keep_their_shape(layer):
    layer.set_weights(torch.zeros(E, F, D), torch.zeros(E, D, F))
    for up, down in ((torch.zeros(E, F + 1, D), torch.zeros(E, D, F + 1)), (torch.zeros(E + 1, F, D), torch.zeros(E + 1, D, F)),
                     (torch.zeros(E, F, D), torch.zeros(E, F, D))):
        with pytest.raises(ValueError):
            layer.set_weights(up, down)
    with pytest.raises(ValueError):
        moe.ExpertFFN(torch.zeros(F, D), torch.zeros(D, F), K)
