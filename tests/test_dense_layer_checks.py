"""What DenseFFN refuses (CPU): the library's calls are replaced by a recorder, so that a check which comes after a call
shows too."""

import pytest
import torch

from sparse_matmul_ffns_amd import dense

D, F = 24, 40


class Called(Exception):
    pass


class Calls:
    def __getattr__(self, name):
        def call(*args, **kw):
            raise Called(name)
        return call

    def _act(self, act):
        if act not in ("none", "relu", "gelu_tanh", "silu"):
            raise ValueError(act)


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    monkeypatch.setattr(dense, "_nm", Calls())


def _layer(**kw):
    return dense.DenseFFN(torch.zeros(D), torch.zeros(F, D), torch.zeros(D, F), **kw)


def test_shapes_of_the_parameters():
    _layer(b_up=torch.zeros(F), b_down=torch.zeros(D))
    for args in ((torch.zeros(F), torch.zeros(F, D), torch.zeros(D, F)), (torch.zeros(D), torch.zeros(F, D), torch.zeros(F, D)),
                 (torch.zeros(D), torch.zeros(1, F, D), torch.zeros(D, F))):
        with pytest.raises(ValueError):
            dense.DenseFFN(*args)
    for kw in (dict(b_up=torch.zeros(D)), dict(b_down=torch.zeros(F)), dict(act="gelu")):
        with pytest.raises(ValueError):
            _layer(**kw)


def test_forward_and_backward():
    layer = _layer(train=True)
    with pytest.raises(Called):
        layer.forward(torch.zeros(5, D))
    for x in (torch.zeros(5, D + 1), torch.zeros(D), torch.zeros(1, 5, D)):
        with pytest.raises(ValueError):
            layer.forward(x)
    with pytest.raises(ValueError):
        _layer().forward(torch.zeros(5, D), return_saved=True)
    with pytest.raises(RuntimeError):
        layer.backward(torch.zeros(5, D))
