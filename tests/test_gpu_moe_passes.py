"""Several passes of one ExpertFFN before their gradients, and inputs that change between the passes (GPU).

The calls are deterministic (an identical call gives identical bits), so every comparison is exact."""

import threading

import pytest
import torch

from sparse_matmul_ffns_amd.moe import ExpertFFN
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
E, D, F, K = 8, 256, 128, 2


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def _layer():
    return ExpertFFN((_rand(1, E, F, D) * 0.1).bfloat16(), (_rand(2, E, D, F) * 0.1).bfloat16(), K, train=True)


def _batch(i, T=40):
    return _rand(10 + i, T, D).bfloat16(), _rand(20 + i, T, E), _rand(30 + i, T, D).bfloat16()


def _alone(i):
    x, logits, dy = _batch(i)
    layer = _layer()
    return layer.forward(x, logits), *layer.backward(dy)


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_micro_batches_with_their_saved_passes():
    layer, want = _layer(), [_alone(i) for i in range(3)]
    passes = [layer.forward(x, logits, return_saved=True) for x, logits, _ in map(_batch, range(3))]
    assert layer.saved is None
    for i in (1, 0, 2, 1):                      # in any order, and again
        y, saved = passes[i]
        assert _same((y, *layer.backward(_batch(i)[2], saved)), want[i])


def test_passes_of_two_threads():
    layer, want, got = _layer(), [_alone(i) for i in range(2)], {}
    met = threading.Barrier(2)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            x, logits, dy = _batch(i)
            met.wait(30)
            y, saved = layer.forward(x, logits, return_saved=True)
            met.wait(30)
            got[i] = (y, *layer.backward(dy, saved))
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert all(_same(got[i], want[i]) for i in range(2))


def test_a_lost_pass_is_refused():
    layer, want = _layer(), _alone(1)
    (x0, l0, dy0), (x1, l1, dy1) = _batch(0), _batch(1)
    layer.forward(x0, l0)
    y1 = layer.forward(x1, l1)
    assert _same((y1, *layer.backward(dy1)), want)
    with pytest.raises(RuntimeError):            # there is no pass of x0 any more
        layer.backward(dy0)
    # an evaluation between the steps, and the same pass again, are no loss
    layer.forward(x0, l0)
    layer.backward(dy0)
    layer.forward(x0, l0)                        # evaluation
    layer.forward(x1, l1)
    assert _same(layer.backward(dy1), want[1:])
    y1 = layer.forward(x1, l1)
    assert _same(layer.backward(dy1), want[1:]) and _same(layer.backward(dy1), want[1:])


def test_changes_between_the_passes_are_refused():
    x, logits, dy = _batch(0)
    for change in (lambda l: x.add_(1), lambda l: logits.zero_(), lambda l: l.set_weights(_rand(3, E, F, D).bfloat16(),
                                                                                         _rand(4, E, D, F).bfloat16())):
        layer = _layer()
        layer.forward(x, logits)
        layer.backward(dy)                       # as it was: fine
        _, saved = layer.forward(x, logits, return_saved=True)
        change(layer)
        for args in ((dy,), (dy, saved)):
            with pytest.raises(RuntimeError):
                layer.backward(*args)
        layer.forward(x, logits)
        layer.backward(dy)


def test_inference_tensors_have_no_version():
    with torch.inference_mode():
        x, logits, dy = _batch(0)
        layer = _layer()
        layer.forward(x, logits)
        layer.backward(dy)


def test_saved_needs_training():
    x, logits, _ = _batch(0)
    layer = ExpertFFN(_rand(1, E, F, D).bfloat16(), _rand(2, E, D, F).bfloat16(), K)
    with pytest.raises(ValueError):
        layer.forward(x, logits, return_saved=True)
