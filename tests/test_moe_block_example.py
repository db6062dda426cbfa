"""The operators together, as examples/moe_block.py runs them: forward and gradients against
the same block in 64-bit torch with autograd, the experts chosen as the library chose them.

Tolerance: every bf16 tensor between two products is rounded once (2^-8 at most, 2^-8 / sqrt(3)
in the root mean square), and at most six of them lie on the way of a result: 6 * 2^-8 / sqrt(3)
in relative L2, under 1.5e-2.
"""

import importlib.util
import os

import pytest
import torch

from tests.conftest import ROOT

REL = 1.5e-2


def example():
    spec = importlib.util.spec_from_file_location(
        "moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rel(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def test_the_example_imports_without_a_gpu():
    assert example().MoEBlock.__doc__


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 48, 700])
def test_block_forward_and_gradients(T):
    ex = example()
    b = ex.MoEBlock(T, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    b.bias.copy_(torch.randn(b.E, generator=g, device="cuda") * 0.05)
    x = torch.randn(T, b.H, generator=g, device="cuda").bfloat16()
    y = b.forward(x)
    dy = torch.randn(T, b.H, generator=g, device="cuda").bfloat16()
    grads = b.backward(x, dy)

    d = lambda t: t.double().requires_grad_(True)
    p = {n: d(getattr(b, n)) for n in grads}
    h = x.double() @ p["w_o"].t() + x.double()
    logits = h @ p["w_r"].t()
    ids = b.ids.long()
    s = torch.sigmoid(logits).gather(1, ids)
    w = s / s.sum(1, keepdim=True)
    hd = h.detach()  # the experts are frozen: nothing flows through their products
    I = b.w_down.shape[2]
    rows = torch.zeros(T, b.K, b.H, dtype=torch.float64, device="cuda")
    for e in range(b.E):
        at = (ids == e).nonzero()
        if len(at):
            gu = hd[at[:, 0]] @ b.w_gate_up[e].double().t()
            a = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
            rows[at[:, 0], at[:, 1]] = a @ b.w_down[e].double().t()
    c = (w[:, :, None] * rows).sum(1)
    z = h @ p["w_1"].t() + p["b_1"]
    ref = torch.nn.functional.silu(z) @ p["w_2"].t() + c
    assert rel(y, ref.detach()) < REL
    assert rel(b.w, w.detach()) < REL
    ref.backward(dy.double())
    for name, grad in grads.items():
        assert rel(grad, p[name].grad) < REL, name


@pytest.mark.gpu
def test_fitting_lowers_the_loss():
    losses = example().fit(T=256, steps=8)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
