"""The operators of a trained block together, as examples/moe_train.py runs them: forward and every
gradient against the same block in 64-bit torch with autograd, the experts chosen as the library
chose them.

Tolerance: every bf16 tensor between two operators is rounded once (2^-8 at most, 2^-8 / sqrt(3) in
the root mean square).  On the longest way, from a parameter before the experts to the output and
back, lie y, z, h, c, s, dout, dc, drows, dh, dz, dy and the result's own rounding: 12 of them, 12 *
2^-8 / sqrt(3) in relative L2 if they all added up, under 2.8e-2.
"""

import importlib.util
import os

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.conftest import ROOT

REL = 2.8e-2


def example():
    spec = importlib.util.spec_from_file_location(
        "moe_train", os.path.join(ROOT, "examples", "moe_train.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rel(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def reference(b, x, params):
    """The block in 64 bits with the library's choice of experts."""
    p, T, I = params, b.T, b.h.shape[1]
    norm = lambda v: v / (v.pow(2).mean(1, keepdim=True) + b.EPS).sqrt()
    y = norm(x) * p["n_1"]
    ids = b.ids.long()
    s = torch.sigmoid(y @ p["w_r"].t()).gather(1, ids)
    w = s / s.sum(1, keepdim=True)
    gate = torch.sigmoid(y @ p["w_g"].t())
    c = torch.zeros_like(y)
    for e in range(b.E):
        t, k = (ids == e).nonzero(as_tuple=True)
        if len(t):
            z = y[t] @ p["w_gu"][e].t()
            h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
            c = c.index_add(0, t, w[t, k][:, None] * (h @ p["w_d"][e].t()))
    s = x + 0.5 * gate * p["scale"] * (norm(c) * p["post"])
    return s, norm(s) * p["n_2"]


def test_the_example_imports_without_a_gpu():
    assert example().TrainedMoEBlock.__doc__


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 48, 700, 3000])
def test_block_forward_and_gradients(T):
    b = example().TrainedMoEBlock(T, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    b.bias.copy_(torch.randn(b.E, generator=g, device="cuda") * 0.05)
    x = torch.randn(T, b.H, generator=g, device="cuda").bfloat16()
    out = b.forward(x).clone()
    dout = torch.randn(T, b.H, generator=g, device="cuda").bfloat16()
    dx = b.backward(x, dout)
    p = {n: t.double().requires_grad_(True) for n, t in b.params.items()}
    xd = x.double().requires_grad_(True)
    s, ref = reference(b, xd, p)
    assert rel(b.s, s.detach()) < REL
    assert rel(out, ref.detach()) < REL
    ref.backward(dout.double())
    assert rel(dx, xd.grad) < REL
    for n, grad in b.grads.items():
        assert rel(grad, p[n].grad) < REL, n
    used = b.counts.cpu()
    for e in range(b.E):
        if used[e] == 0:
            assert (b.grads["w_gu"][e] == 0).all() and (b.grads["w_d"][e] == 0).all()
    kept = {n: t.clone() for n, t in b.grads.items()}
    want = sum(float(t.double().pow(2).sum()) for t in kept.values()) ** 0.5
    norm = b.step(0.0, 0.5 * want)
    assert abs(norm.item() / want - 1) < 1e-6
    for n, t in b.grads.items():
        assert rel(t, 0.5 * kept[n].double()) < 2.0 ** -8
    moe.sync_check()


@pytest.mark.gpu
def test_a_captured_step_replays():
    """Forward and backward captured into one graph, replayed on other tokens."""
    b = example().TrainedMoEBlock(300, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dout = (torch.randn(300, b.H, generator=g, device="cuda").bfloat16() for _ in range(2))
    b.backward(b.forward(x), dout)  # warm-up: sizes and limits are set up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(x)
        dx = b.backward(x, dout)
        moe.clip_grad_norm(b.list, 1e-3, b.norm, b.clip_ws)
    x.copy_(torch.randn(300, b.H, generator=g, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    got = {n: t.clone() for n, t in b.grads.items()}
    got_dx, got_out, got_norm = dx.clone(), b.out.clone(), b.norm.clone()
    out = b.forward(x)
    want_dx = b.backward(x, dout)
    moe.clip_grad_norm(b.list, 1e-3, b.norm, b.clip_ws)
    assert torch.equal(got_out, out) and torch.equal(got_dx, want_dx)
    assert torch.equal(got_norm, b.norm)
    for n, t in b.grads.items():
        assert torch.equal(got[n], t), n


@pytest.mark.gpu
def test_fitting_runs():
    log = example().fit(T=200, steps=3)
    assert len(log) == 3 and all(l == l and n > 0 for l, n in log)
