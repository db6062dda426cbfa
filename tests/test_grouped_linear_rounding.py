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


@pytest.mark.parametrize("sizes", [[9, 0, 20], [70, 50]], ids=str)
@pytest.mark.parametrize("fin,fout", [(14336, 64), (4096, 200)])
def test_float32_sums_leave_the_tensor_core_every_256_values(sizes, fin, fout):
    """Values of one sign, whose truncated additions add up in the mean error of the results (their own
    roundings, 2^-25 each, average out).  The linear layers leave 1.4e-8 with 256 values and 7.3e-7
    with 1024; the limit lies between, as in test_linear_accumulation.  (Over 64 rows a group they leave
    it every 512.)"""
    c = Case(sizes, fin, fout, False, out=F32, seed=32)
    c.x.copy_(torch.rand(c.x.shape, device="cuda") + 0.5)
    c.w.copy_(torch.rand(c.w.shape, device="cuda") + 0.5)
    y, _ = c.forward()
    for e, at, w in c.groups():
        want = c.x[at].double() @ w.t()
        rel = (y[at].double() - want) / want
        assert abs(rel.mean().item()) < 1.5e-7
    d = Case(sizes, fout, fin, False, dx=F32, seed=33)  # the reduction of dx: over outputs
    d.dy.copy_(torch.rand(d.dy.shape, device="cuda") + 0.5)
    d.w.copy_(torch.rand(d.w.shape, device="cuda") + 0.5)
    dx, _ = d.backward(want_dw=False)
    for e, at, w in d.groups():
        want = d.dy[at].double() @ w
        rel = (dx[at].double() - want) / want
        assert abs(rel.mean().item()) < 1.5e-7
    moe.sync_check()


@pytest.mark.parametrize("want_dx", [True, False])
@pytest.mark.parametrize("sizes", [[16] * 6, [16, 0, 9], [200, 90], [20] * 9 + [0, 250]], ids=str)
@pytest.mark.parametrize("fin,fout", [(320, 256), (333, 201)])
def test_dw_is_off_by_little_more_than_its_own_rounding(sizes, fin, fout, want_dx):
    """With a float32 dx dz keeps 16 bits, for dw as well.  Element by element half a step of the
    result and (PARTS + FAST + ACC) of S; in L2 what rounding the exact dw leaves (some 1e5
    elements, whose mean square moves by less than a hundredth; a twentieth is allowed) and the
    same share of S.  A dz rounded to bf16 would add as much again as the result's own rounding, in
    the mean square: 41% in L2."""
    c = Case(sizes, fin, fout, True, dx=F32, pad=0 if fin == 320 else 3, tail=3, seed=34)
    dx, dw = c.backward(want_dx=want_dx)
    err = own = share = 0.0
    for e, at, w in c.groups():
        d, x = c.dz(at), c.x[at].double()
        ref, S = d.t() @ x, d.t().abs() @ x.abs()
        off = S * (acc(x.shape[0], BF16) + PARTS + FAST)
        got = dw[e * c.N:(e + 1) * c.N, :fin].double()
        assert_close(got, ref, off * (1 + 2.0 ** -8) + ref.abs() * 2.0 ** -8 + 1e-37)
        err += ((got - ref) ** 2).sum().item()
        own += ((ref.to(BF16).double() - ref) ** 2).sum().item()
        share += (off ** 2).sum().item()
    assert err ** 0.5 <= 1.05 * own ** 0.5 + share ** 0.5
    if want_dx:
        c.check_backward(dx, dw)
    moe.sync_check()


@pytest.mark.parametrize("sizes", [[16] * 6, [60, 0, 40], [300, 90], [3000]], ids=str)
@pytest.mark.parametrize("fin,fout", [(320, 768), (333, 201)])
def test_a_float32_dx_keeps_the_bits_of_dz(sizes, fin, fout):
    """In relative L2: the float32 results' own rounding (2^-24), three parts' (2^-24) and the fast
    exponential (some 2^-22 of a term, in sums of hundreds of them of either sign) stay below 3e-7,
    the truncating accumulators, drained every 256 values, below 9e-7: 2.3e-7 for one product of 2048
    values, and three share one here.  The limit is 1e-6; two parts would leave 2.2e-6 alone."""
    c = Case(sizes, fin, fout, True, dx=F32, pad=0 if fin == 320 else 3, tail=3, seed=35)
    dx, _ = c.backward()
    err = size = 0.0
    for e, at, w in c.groups():
        want = c.dz(at) @ w
        err += ((dx[at, :fin].double() - want) ** 2).sum().item()
        size += (want ** 2).sum().item()
    assert (err / size) ** 0.5 < 1e-6
    moe.sync_check()
