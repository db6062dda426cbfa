"""Clipping with an infinite largest norm, and norms that are not finite: include/moe.h's rules.

The factor is grad_scale where max_norm is infinite, whatever the norm (infinite over infinite would
be NaN in every result); a norm that is NaN makes every result NaN; an infinite norm makes the factor
0 under a finite max_norm.  Factors are powers of two here, so every product is exact.
"""

import math

import pytest
import torch

from tests.test_clip_grad_norm import BF16, F32, clip, make

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("tensors", [2, 70])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [INF, -INF])
def test_an_infinite_gradient_without_a_limit(value, dtype, tensors):
    grads = make([5000] + [20] * (tensors - 1), (dtype,), seed=4)
    grads[0][4321] = value
    outs = [torch.empty_like(g) for g in grads]
    norm = clip(grads, outs, INF, scale=0.5)
    assert norm.item() == INF
    for g, o in zip(grads, outs):
        assert torch.equal(o, g * 0.5)
    kept = [g.clone() for g in grads]
    clip(grads, grads, INF)  # in place, factor 1: nothing changes
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))


@pytest.mark.parametrize("max_norm", [1.0, INF])
def test_a_gradient_that_is_nan(max_norm):
    grads = make([5000, 20], (F32,), seed=5)
    grads[0][17] = float("nan")
    grads[1][3] = INF
    outs = [torch.zeros_like(g) for g in grads]
    assert math.isnan(clip(grads, outs, max_norm).item())
    assert all(torch.isnan(o).all() for o in outs)


def test_an_infinite_gradient_under_a_limit():
    grads = make([5000, 20], (F32,), seed=6)
    grads[0][17] = INF
    outs = [torch.ones_like(g) for g in grads]
    assert clip(grads, outs, 1.0).item() == INF
    assert torch.isnan(outs[0][17]) and (outs[1] == 0).all()
    outs[0][17] = 0
    assert (outs[0] == 0).all()


def test_no_gradient_at_all_without_a_limit():
    grads = [torch.zeros(100, device="cuda")]
    outs = [torch.ones(100, device="cuda")]
    assert clip(grads, outs, INF, eps=0.0).item() == 0
    assert (outs[0] == 0).all()
