"""Linear layers at the ends of their numerics: the largest float32 values.

The formulas in 64 bits and the tolerances' terms are those of tests/test_linear.py.
"""

import math

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_linear import config, workspace

FLT_MAX = torch.finfo(torch.float32).max


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------- the largest float32 values ----

@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 8, 9, 40, 300])
@pytest.mark.parametrize("pad", [0, 3])
def test_the_largest_finite_values_stay_finite(rows, pad):
    """bf16 ends at 3.39e38 and float32 at 3.40e38: the values between have three parts too."""
    fin, fout = 72, 56
    g = gen(rows + pad)
    x = torch.randn(rows, fin + pad, generator=g, device="cuda")
    big = torch.tensor([FLT_MAX, -FLT_MAX, 3.3961e38, -3.4e38], device="cuda")
    at = torch.arange(rows, device="cuda")
    x[at, at % fin] = big[at % 4]
    w = torch.randn(fout, fin, generator=g, device="cuda") * 1e-2
    b = torch.randn(fout, generator=g, device="cuda")
    c = config(rows, fin, fout, dtype=moe.F32, x_stride=fin + pad)
    y = torch.empty(rows, fout, device="cuda")
    moe.linear(c, x, w, b, None, y, None, workspace(c))
    moe.sync_check()
    xd = x[:, :fin].double()
    want = xd @ w.double().t() + b.double()
    size = xd.abs() @ w.double().abs().t()
    adds = 6 * math.ceil(fin / 16) + 16
    tol = (adds * 2.0 ** -23 + 8 * 2.0 ** -24) * size + 2.0 ** -24 * 1.01 * want.abs() + 1e-6
    assert torch.isfinite(y).all()
    assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_gradients_of_the_largest_finite_values_stay_finite(rows):
    fin, fout = 72, 56
    g = gen(rows)
    x = torch.randn(rows, fin, generator=g, device="cuda") * 1e-2
    w = torch.randn(fout, fin, generator=g, device="cuda") * 1e-2
    dy = torch.randn(rows, fout, generator=g, device="cuda")
    at = torch.arange(min(rows, fout), device="cuda")
    dy[at, at] = torch.where(at % 2 == 0, FLT_MAX, -FLT_MAX)
    c = config(rows, fin, fout, dtype=moe.F32)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    moe.linear_backward(c, dy, x, w, None, dx, dw, None, workspace(c))
    moe.sync_check()
    d = dy.double()
    for got, want, size, depth in ((dx, d @ w.double(), d.abs() @ w.double().abs(), fout),
                                   (dw, d.t() @ x.double(), d.abs().t() @ x.double().abs(), rows)):
        adds = 6 * math.ceil(min(depth, 128) / 16) + depth / 128 + 16
        tol = (adds * 2.0 ** -23 + 8 * 2.0 ** -24) * size + 2.0 ** -24 * 1.01 * want.abs() + 1e-6
        assert torch.isfinite(got).all()
        assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.gpu
def test_infinities_and_nan_still_reach_their_outputs_only():
    rows, fin, fout = 40, 72, 56
    x = torch.randn(rows, fin, generator=gen(2), device="cuda")
    x[3, 5], x[7, 0], x[9, 71] = float("inf"), float("-inf"), float("nan")
    w = torch.randn(fout, fin, generator=gen(3), device="cuda")
    c = config(rows, fin, fout, dtype=moe.F32)
    y = torch.empty(rows, fout, device="cuda")
    moe.linear(c, x, w, None, None, y, None, workspace(c))
    moe.sync_check()
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[[3, 7, 9]] = True
    assert not torch.isfinite(y[bad]).any() and torch.isfinite(y[~bad]).all()
