"""What the feed-forward layer does with inputs that are not plain [tokens, features] values."""
import pytest
import torch

from gpu_util import DEV
from test_gpu_feedforward import build

pytestmark = pytest.mark.gpu


def test_inputs_of_another_shape_are_refused():
    wb, gamma, beta, ff, g = build(256, 384, 12, 1)
    x = torch.randn(12, 256, generator=g, device=DEV).to(torch.bfloat16)
    ff.forward(x)
    for bad in (x[:1], x[0], x[:, :1], x[None], x[:11], x.t()):
        with pytest.raises(ValueError, match=r"\[12, 256\]"):
            ff.forward(bad)
        with pytest.raises(ValueError, match=r"\[12, 256\]"):
            ff.backward(bad)


def test_inputs_that_require_gradients():
    """The layer's buffers stay plain storage: no graph hangs on them from step to step, and the
    results are those of the same values without a graph."""
    wb, gamma, beta, ff, g = build(256, 384, 12, 2)
    x = torch.randn(12, 256, generator=g, device=DEV).to(torch.bfloat16)
    want, dx = ff.forward(x).clone(), ff.backward(x).clone()
    leaf = x.clone().requires_grad_()
    for _ in range(2):
        y = ff.forward(leaf * 1.0)
        assert not y.requires_grad and not ff.x.requires_grad and ff.x.grad_fn is None
        assert torch.equal(y, want)
        got = ff.backward(leaf * 1.0)
        assert not got.requires_grad and ff.dy.grad_fn is None
        assert torch.equal(got, dx)
