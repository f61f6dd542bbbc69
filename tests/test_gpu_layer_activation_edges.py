"""Gradients of mxfp8_act_backward on the GPU for gates and GELU inputs as large as a checkpoint
holds.

Tolerance: 2^-21 (6 + |w|) of the terms as in test_gpu_layer_activation.py, with |w|, the sigmoid's
argument, counted up to 90: further out the exponential is under 2^-129 and the function is its
asymptote, so that no error grows with the argument any more.  A sigmoid (or 1 minus it) below 2^-125
may count as 0, which costs its term 2^-125 of the other factors, the argument counted up to 90 there
too: x e^-x falls from then on."""
import pytest
import torch

import layer_reference as R
from gpu_util import DEV, require_gpu
from mxfp8_block_scaled_partial_amd import layer as L

pytestmark = pytest.mark.gpu


def column(code, scale):
    """[n, 1] values, each in a block of its own: code * 2^(scale - 127)."""
    d = torch.tensor(code, dtype=torch.uint8, device=DEV).view(-1, 1)
    s = torch.tensor(scale, dtype=torch.uint8, device=DEV).view(-1, 1)
    return d, s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("func", ["gelu", "swiglu"])
def test_gradients_of_far_out_inputs(func, dtype):
    """Inputs +-1.75 * 2^e for e from 0 to 127, where c = 1 - s of a large positive gate must vanish
    faster than the gate grows."""
    require_gpu()
    exponents = list(range(-3, 128))
    code = [0x7E if i % 2 == 0 else 0xFE for i in range(2 * len(exponents))]  # +-1.75 * 2^8
    scale = [e - 8 + 127 for e in exponents for _ in range(2)]
    saved = [column(code, scale)]
    if func == "swiglu":  # up: +-1 and +-2.5 in turn
        saved.append(column([(0x38, 0xB8, 0x42, 0xC2)[i // 2 % 4] for i in range(len(code))], [127] * len(code)))
    d = torch.tensor([1.0, -0.25], dtype=dtype, device=DEV).repeat(len(exponents)).view(-1, 1).contiguous()
    out = [torch.empty_like(d) for _ in saved]
    L.mxfp8_act_backward(L.make_act(func, grad=d, saved=saved, out=out))
    u = [R.decode(*s, 1, 128) for s in saved]
    w = u[0] if func == "swiglu" else 2 * R.W * (u[0] + 0.044715 * u[0] ** 3)
    far = w.abs().clamp(max=90.0)
    b = u[1].abs() if func == "swiglu" else torch.ones_like(w)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for i, (y, terms) in enumerate(R.act_gradients(func, u, d.double())):
        # far out the float64 formula of GELU's derivative overflows into 0 * inf: it is d * step(u)
        step = d.double() * (u[0] > 0)
        if func == "gelu":
            y = torch.where(w.abs() > 700, step, y)
            terms = torch.where(w.abs() > 700, d.double().abs(), terms)
        # da's terms have d, b and the argument beside the sigmoid; db's d and the gate itself, which
        # the sigmoid of a negative gate takes to 0 like the argument
        tol = 2.0 ** -21 * (6 + far) * terms + 2.0 ** -125 * d.double().abs() * (1 + far) ** 3 * (1 + b)
        assert ((out[i].double() - y).abs() <= half * (y.abs() + tol) + tol).all(), i
