"""mxfp8_layernorm_forward on the GPU where a row's mean is far above its deviation, and for rows of
millions of columns.

Tolerances, with d = x - mean, m = mean |x|, a = mean |d| and s the deviation, all in float64.  A
row's sums add at most 32 values serially in a lane and a tree of 10 above it, or (rows past the
registers) 8 in a tree under a compensated sum: 42 roundings of 2^-24 < 2^-18.  So a first mean is off
by e <= 2^-18 m, and the sum of the deviations from it brings that down to 2^-18 (e + a), beside the
rounding of each deviation, 2^-24 (|d| + e).  The variance, taken from those deviations and corrected
by e^2, is within 2^-18 (s^2 + 2 e^2), rstd within half of that, and xh takes its product's 4
roundings.  The stored mean is rounded once more, 2^-24 |mean|."""
import pytest
import torch

from gpu_util import DEV, require_gpu
from mxfp8_block_scaled_partial_amd import layer as L

pytestmark = pytest.mark.gpu


def check(x):
    rows = x.shape[0]
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    L.mxfp8_layernorm_forward(L.make_layernorm(x, y=y, mean=mean, rstd=rstd, eps=0.0))
    for r in range(rows):
        v = x[r].double()
        mu, m = v.mean(), v.abs().mean()
        d = v - mu
        a, var = d.abs().mean(), d.square().mean()
        e = 2.0 ** -18 * m
        off = 2.0 ** -18 * (e + a)
        assert (mean[r].double() - mu).abs() <= off + 2.0 ** -24 * mu.abs()
        rel = 2.0 ** -18 * (1 + 2 * e * e / var) + 2.0 ** -22
        assert (rstd[r].double() * var.sqrt() - 1).abs() <= rel
        xh = d / var.sqrt()
        tol = (off + 2.0 ** -24 * (d.abs() + e)) / var.sqrt() + (rel + 2.0 ** -22) * xh.abs()
        assert ((y[r].double() - xh).abs() <= tol).all()


@pytest.mark.parametrize("ratio", [1e3, 1e5])
@pytest.mark.parametrize("size", [(9, 129), (40, 1001), (17, 5000), (3, 16384), (3, 40001)], ids=str)
def test_mean_far_above_the_deviation(size, ratio):
    require_gpu()
    g = torch.Generator(device=DEV).manual_seed(size[1])
    x = ratio * (1 + torch.rand(size[0], 1, generator=g, device=DEV)) + torch.randn(*size, generator=g, device=DEV)
    check(x)


def test_rows_of_millions_of_columns():
    """Values a little above 1: each addition to a long serial sum would round the same way."""
    require_gpu()
    g = torch.Generator(device=DEV).manual_seed(3)
    check(1.0003 + 1e-4 * torch.randn(2, 1 << 24, generator=g, device=DEV))


def test_backward_of_millions_of_columns():
    """dx of a wide row: its two sums are as exact as the forward pass's.  mean(g) and mean(g xh) are
    within 2^-18 of their terms' mean magnitude; dx is a few roundings away from that."""
    require_gpu()
    g = torch.Generator(device=DEV).manual_seed(4)
    cols = 1 << 24
    x = torch.randn(1, cols, generator=g, device=DEV)
    dy = 1.0003 + 1e-4 * torch.randn(1, cols, generator=g, device=DEV)
    m = x.double().mean(1).float()
    r = (1 / x.double().var(1, unbiased=False).sqrt()).float()
    dx = torch.empty_like(x)
    L.mxfp8_layernorm_backward(L.make_layernorm(x, mean=m, rstd=r, dy=dy, dx=dx))
    xh, d = (x.double() - m.double()) * r.double(), dy.double()
    m1, m2 = d.mean(), (d * xh).mean()
    want = r.double() * (d - m1 - xh * m2)
    tol = r.double() * (2.0 ** -18 * (d.abs().mean() + xh.abs() * (d * xh).abs().mean()) +
                        2.0 ** -22 * (d.abs() + (xh * m2).abs()))
    assert ((dx.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("cols", [300, 5000, 40001])
def test_statistics_of_rows_that_are_not_finite(cols):
    """The mean of a row with an infinity is that infinity, of one with both or a NaN NaN; rows whose
    squares overflow have rstd 0."""
    require_gpu()
    inf = float("inf")
    x = torch.randn(6, cols, device=DEV)
    x[0, 7], x[1, cols - 1], x[2, 3], x[2, 50], x[3, 11] = inf, -inf, inf, -inf, float("nan")
    x[4] = 1e30 * x[4]
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    L.mxfp8_layernorm_forward(L.make_layernorm(x, y=y, mean=mean, rstd=rstd))
    assert mean[0] == inf and mean[1] == -inf and mean[2:4].isnan().all() and mean[4:].isfinite().all()
    assert rstd[:4].isnan().all() and rstd[4] == 0 and rstd[5].isfinite()
    assert y[:4].isnan().all() and (y[4] == 0).all() and y[5].isfinite().all()
