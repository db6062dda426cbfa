"""How far the gradients of a grouped bf16 SwiGLU layer are from the definition, beyond the rounding of
the results themselves.

A half step of bf16 is 2^-8 of the value, of what two bf16 parts hold 2^-17.  silu and its slope are
computed with the hardware's exponential and reciprocal: FAST = 1e-5 of their size (the slope's series
near its zero is good to 2e-6 there; elsewhere 1 + z q loses no more than a factor of 5).  S is a
sum's terms in absolute value; a tensor core's sum of n products is off by ACC(n) S, as in
test_grouped_linear.
"""

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_grouped_linear import BF16, F32, Case, acc, assert_close

pytestmark = pytest.mark.gpu

FAST = 1e-5
PARTS = 2.0 ** -17


def test_the_slope_keeps_its_accuracy_near_its_zero():
    """dx is the gate's dz itself: its weights are the unit matrix, those of up are zero."""
    n, rows = 64, 96
    c = Case([rows], n, n, True, dx=F32, seed=31)
    c.w.zero_()
    c.w[:n] = torch.eye(n, device="cuda")
    # the bf16 numbers around -1.2785, each in every row; a step is 2^-7 there
    z = (-1.2785 + (torch.arange(n, device="cuda") - n // 2) * 2.0 ** -7).to(BF16)
    c.z[:, :n] = z
    dx, _ = c.backward(want_dw=False)
    g = z.double()
    s = torch.sigmoid(g)
    want = c.dy.double() * c.z[:, n:].double() * (s * (1 + g * (1 - s)))
    assert_close(dx, want, want.abs() * (PARTS + FAST) + 1e-37)
    moe.sync_check()
