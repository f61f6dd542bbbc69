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
