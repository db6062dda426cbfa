"""Linear layers at the ends of their numerics: the largest float32 values and the
activations' tails.

The formulas in 64 bits and the tolerances' terms are those of tests/test_linear.py.
"""

import math

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_linear import act, config, slope, workspace

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


# ------------------------------------------------------------- the activations' tails ----

def grid(lo, hi):
    """Every bf16 value of lo..hi, in rows of 64."""
    v = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v) & (v >= lo) & (v <= hi) & (v.abs() >= 2.0 ** -20)]
    return v[: v.numel() // 64 * 64].reshape(-1, 64).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("a", [moe.ACT_GELU, moe.ACT_GELU_TANH, moe.ACT_SILU])
@pytest.mark.parametrize("few", [True, False])
def test_bf16_activations_are_rounded_once_over_their_whole_range(a, few):
    """Through an identity, so that z is the input: the value's own error is a few units in the
    last place of float32 and of the exponential's argument (under 2^-14 of its size down to the
    smallest normal numbers), then comes the one rounding."""
    x = grid(-12.9, 12.9)
    x = x[:8 * (x.shape[0] // 8)]
    eye = torch.eye(64, device="cuda").bfloat16()
    parts = x.reshape(-1, 1, 64) if few else x.reshape(1, -1, 64)
    for xs in parts:
        for f32 in (False, True):
            c = config(xs.shape[0], 64, 64, activation=a, out_dtype=moe.F32 if f32 else moe.BF16)
            y = torch.empty(xs.shape, device="cuda", dtype=torch.float32 if f32 else xs.dtype)
            moe.linear(c, xs.contiguous(), eye, None, None, y, None, workspace(c))
            want = act(a, xs.double())
            tol = (2.0 ** -14 + (0.0 if f32 else 2.0 ** -8)) * want.abs() + 2.0 ** -122
            if f32:
                tol = tol + 2.0 ** -22 * xs.double().abs() * (xs > -1.0)
            assert ((y.double() - want).abs() <= tol).all()
    moe.sync_check()


@pytest.mark.gpu
@pytest.mark.parametrize("a", [moe.ACT_GELU, moe.ACT_GELU_TANH, moe.ACT_SILU])
def test_bf16_slopes_in_the_tail_are_rounded_once(a):
    """dz through an identity: dy act'(z), rounded to bf16, exactly the gradient.  Below -3 every
    slope is away from its zero and its terms do not cancel by more than a factor of three."""
    z = grid(-12.5, -3.0)
    eye = torch.eye(64, device="cuda").bfloat16()
    dy = torch.ones_like(z)
    c = config(z.shape[0], 64, 64, activation=a)
    dx = torch.empty_like(z)
    moe.linear_backward(c, dy, None, eye, z, dx, None, None, workspace(c))
    moe.sync_check()
    want = slope(a, z.double())
    assert ((dx.double() - want).abs() <= (2.0 ** -12 + 2.0 ** -8) * want.abs() + 2.0 ** -118).all()
