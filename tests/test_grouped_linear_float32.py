"""Both gradients of a float32 grouped layer run in one launch: each is bit for bit what it is by
itself, on one stream, on two at once and replayed from a graph, with launches of other calls around
it.  Tolerances are those of test_grouped_linear.
"""

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_grouped_linear import F32, Case

pytestmark = pytest.mark.gpu

# fewer tiles than SMs; more; a group of none; one group; odd sizes
LAYERS = [([100, 0, 33, 7], 128, 64), ([700, 900, 0, 1100], 512, 512), ([5], 64, 64),
          ([129, 3, 0, 260], 333, 201)]


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("sizes,fin,fout", LAYERS, ids=str)
def test_gradients_alone_are_what_they_are_together(sizes, fin, fout, act):
    c = Case(sizes, fin, fout, act, dtype=F32, tail=3, seed=21)
    dx, dw = c.backward()
    c.check_backward(dx, dw)
    for _ in range(3):
        assert torch.equal(c.backward(want_dw=False)[0], dx)
        assert torch.equal(c.backward(want_dx=False)[1], dw)
        again = c.backward()
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    moe.sync_check()


def test_two_streams_at_once():
    cases = [Case(s, i, o, True, dtype=F32, seed=22 + k) for k, (s, i, o) in enumerate(LAYERS[:2])]
    want = [(c.forward(), c.backward()) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        got = [(c.forward(stream=s), c.backward(stream=s)) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))
    moe.sync_check()


def test_operands_written_by_the_kernel_before_the_call():
    """The call's first kernel may be launched while that one still runs."""
    c = Case([300, 0, 129, 70], 256, 128, True, dtype=F32, seed=24)
    other = Case([300, 0, 129, 70], 256, 128, True, dtype=F32, seed=25)
    sets = [[t.clone() for t in (k.x, k.dy, k.z, k.w, k.offsets)] for k in (c, other)]
    want = [k.backward() for k in (c, other)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    places = (c.x, c.dy, c.z, c.w, c.offsets)
    with torch.cuda.graph(graph, stream=stream):
        outs = []
        for s in sets:
            for a, b in zip(places, s):
                a.copy_(b)
            outs.append(c.backward())
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
