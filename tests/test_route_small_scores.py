"""Weights and gradients of logistic scores far below the largest one of a token (chosen for
their bias): they are small, but no smaller than float32 can hold.  Tolerances as in
tests/test_route_scored.py, relative to each value."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_route_scored import G_RTOL, W_RTOL, check, gen, grad, reference_grad

ROWS = [
    (-50.0, -88.0, -95.0, -110.0), (-59.9, -87.5, -89.0, -120.0), (-59.9, -60.1, -90.0, -100.0),
    (-61.0, -90.0, -100.0, -125.0), (-20.0, -60.0, -80.0, -86.0), (3.0, -60.0, -30.0, 90.0),
    (0.0, -1.0, -40.0, -68.0), (-1.0, -1.0, -1.0, -69.0), (100.0, 89.0, 20.0, -60.0),
]


def rows():
    logits = torch.full((len(ROWS), 40), -float("inf"), device="cuda")
    logits[:, [3, 11, 12, 37]] = torch.tensor(ROWS, device="cuda")
    bias = torch.randn(40, generator=gen(1), device="cuda")
    return logits, bias


@pytest.mark.gpu
@pytest.mark.parametrize("with_bias", [True, False])
def test_small_weights_are_kept(with_bias):
    logits, bias = rows()
    c = moe.RouteConfig.make(len(ROWS), 40, 4, score=moe.SCORE_SIGMOID)
    _, w = check(c, logits, bias if with_bias else None)
    assert (w > 0).all()


@pytest.mark.gpu
def test_small_gradients_are_kept():
    logits, bias = rows()
    for scale in (1.0, 2.5):
        c = moe.RouteConfig.make(len(ROWS), 40, 4, score=moe.SCORE_SIGMOID, scale=scale)
        ids, _ = check(c, logits, bias)
        dw = torch.rand(len(ROWS), 4, generator=gen(2), device="cuda") + 0.5
        dw[:, 1::2] *= -3.0  # no term is cancelled by the weighted mean
        got = grad(c, logits, ids, dw).double().cpu().numpy()
        want = reference_grad(c, logits.double().cpu().numpy(), ids.cpu().numpy(),
                              dw.double().cpu().numpy())
        # the factor dw - mean is off by G_RTOL of the largest |dw|, which is under 20 times it
        far = np.abs(want) < 1e-3 * np.abs(want).max(axis=1, keepdims=True)
        np.testing.assert_allclose(got[far], want[far], rtol=20 * G_RTOL, atol=1e-30)
        np.testing.assert_allclose(got, want, rtol=20 * G_RTOL,
                                   atol=G_RTOL * scale * float(dw.abs().max()))
