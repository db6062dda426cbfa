"""The norm over many gradients and clipping, against 64-bit torch.

Tolerances.  Eight squares are added in float32 (8 roundings of 2^-24 at most, so 4 of the norm's),
everything after that in more bits, and the norm is rounded once: 5 2^-24.  The factor is computed
in 64 bits and rounded, a result is a float32 product, rounded once more to its type.
"""

import ctypes
import math

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe

OK, INVALID, WORKSPACE, MISALIGNED = 0, 1, 3, 7
BF16, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24


def step(dtype):
    return 2.0 ** -8 if dtype == BF16 else E


def make(sizes, dtypes, std=1.0, seed=0, shift=0):
    """Gradients, each `shift` elements into its storage."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n + shift, generator=g, device="cuda") * std).to(dtypes[i % len(dtypes)])[
        shift:] for i, n in enumerate(sizes)]


def reference(grads, scale, max_norm, eps):
    norm = scale * math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    return norm, scale * min(1.0, max_norm / (norm + eps))


def clip(grads, outs, max_norm, scale=1.0, eps=1e-6, **kw):
    lst = moe.GradList(grads, outs)
    ws = torch.full((moe.clip_grad_norm_workspace_size(lst),), 255, dtype=torch.uint8,
                    device="cuda")
    norm = torch.full((1,), -1.0, device="cuda")
    moe.clip_grad_norm(lst, max_norm, norm, ws, scale, eps, **kw)
    return norm


def check(grads, outs, norm, max_norm, scale=1.0, eps=1e-6):
    want, factor = reference(grads, scale, max_norm, eps)
    assert abs(norm.item() - want) <= 5 * E * want
    # the factor: eps aside it moves with the norm
    for g, o in zip(grads, outs or []):
        ref = g.double() * factor
        tol = ref.abs() * (6 * E + E + step(o.dtype)) + 2.0 ** -149
        assert ((o.double() - ref).abs() <= tol).all()


SIZES = {
    "one": [1], "few": [3, 0, 17, 1000], "odd": [32768, 32769, 32767, 5, 100001],
    "many": [1 + 37 * i % 2000 for i in range(1300)], "large": [5_000_000, 12345],
    "batch": [64] * 512, "batch and one": [64] * 513,
}


@pytest.mark.gpu
@pytest.mark.parametrize("max_norm", [1.0, 1e6, float("inf")])
@pytest.mark.parametrize("dtypes,outs", [((F32,), F32), ((BF16,), BF16), ((BF16, F32), F32),
                                         ((F32, BF16), BF16)])
@pytest.mark.parametrize("sizes", list(SIZES.values()), ids=list(SIZES))
def test_results_elsewhere(sizes, dtypes, outs, max_norm):
    for shift in (0, 1):
        grads = make(sizes, dtypes, seed=1, shift=shift)
        res = [torch.full((g.numel() + 1,), 7.0, dtype=outs, device="cuda") for g in grads]
        norm = clip(grads, [r[:-1] for r in res], max_norm, scale=0.5)
        check(grads, [r[:-1] for r in res], norm, max_norm, scale=0.5)
        assert all(r[-1] == 7 for r in res)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place_and_alone(dtype):
    grads = make([100, 7, 65536, 40000], (dtype,), seed=2)
    kept = [g.clone() for g in grads]
    norm = clip(grads, None, 1.0)
    check(kept, None, norm, 1.0)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    check(kept, grads, clip(grads, grads, 1.0), 1.0)
    # below the limit now: nothing changes any more
    kept = [g.clone() for g in grads]
    clip(grads, grads, 2.0)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    res = [torch.zeros_like(g) for g in grads]
    lst = moe.GradList(grads, res)
    lst.array[1].out = None  # one tensor without a result
    ws = torch.empty(moe.clip_grad_norm_workspace_size(lst), dtype=torch.uint8, device="cuda")
    moe.clip_grad_norm(lst, 2.0, None, ws)
    assert (res[1] == 0).all() and torch.equal(res[2], grads[2])


@pytest.mark.gpu
@pytest.mark.parametrize("std", [1e-30, 1e-22, 1e18, 1e25, 3e37])
def test_squares_outside_the_range_of_float(std):
    grads = make([1000, 33], (F32, BF16), std=std / 8, seed=3)
    outs = [torch.empty_like(g) for g in grads]
    norm = clip(grads, outs, 1.0)
    check(grads, outs, norm, 1.0)


@pytest.mark.gpu
def test_values_that_are_not_finite():
    for value, factor_is_nan in ((float("nan"), True), (float("inf"), False)):
        grads = make([5000, 20], (F32,), seed=4)
        grads[0][4321] = value
        outs = [torch.empty_like(g) for g in grads]
        norm = clip(grads, outs, 1.0)
        assert not math.isfinite(norm.item())
        if factor_is_nan:
            assert all(torch.isnan(o).all() for o in outs)
        else:
            assert (outs[1] == 0).all() and torch.isnan(outs[0][4321])


@pytest.mark.gpu
def test_nothing_at_all():
    assert clip([], None, 1.0).item() == 0
    assert clip(make([0, 0], (F32,)), None, 1.0).item() == 0
    zeros = [torch.zeros(100, device="cuda")]
    outs = [torch.ones(100, device="cuda")]
    assert clip(zeros, outs, 1.0, eps=0.0).item() == 0
    assert (outs[0] == 0).all()


@pytest.mark.gpu
def test_same_bits_again_captured_and_on_two_streams():
    grads = make([70000, 3, 123457], (BF16, F32), seed=5)
    outs = [torch.empty_like(g) for g in grads]
    first = clip(grads, outs, 1.0)
    want = [o.clone() for o in outs]
    torch.cuda.synchronize()
    lst = moe.GradList(grads, outs)
    ws = torch.empty(moe.clip_grad_norm_workspace_size(lst), dtype=torch.uint8, device="cuda")
    norm = torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.clip_grad_norm(lst, 1.0, norm, ws)
    del lst  # the list was read at capture
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, first) and all(torch.equal(a, b) for a, b in zip(outs, want))
    sets = [(make([50000, 11], (F32,), seed=s), torch.cuda.Stream()) for s in (6, 7)]
    torch.cuda.synchronize()
    keep = []
    for g, s in sets:
        with torch.cuda.stream(s):
            o = [torch.empty_like(t) for t in g]
            keep.append((g, o, clip(g, o, 3.0)))
    torch.cuda.synchronize()
    for g, o, n in keep:
        check(g, o, n, 3.0)


# ---------------------------------------------------------------------- refusals (CPU) ----

A = 0x7000_0000_0000  # never dereferenced: every call below fails validation first


def test_bad_lists_in_the_binding():
    a, b = torch.zeros(4), torch.zeros(5)
    for grads, outs in (([a], [b]), ([a], [a, a]), ([torch.zeros(4, 4).t()], None),
                        ([torch.zeros(3, dtype=torch.float64)], None),
                        ([a], [torch.zeros(4, dtype=torch.float16)])):
        with pytest.raises(ValueError):
            moe.GradList(grads, outs)


@pytest.mark.gpu
def test_results_that_overlap_are_refused():
    flat = torch.zeros(100, device="cuda")
    a, b = flat[:40], flat[40:80]
    x, y = torch.zeros(40, device="cuda"), torch.zeros(40, device="cuda")
    for grads, outs in (([x, y], [a, flat[39:79]]), ([x, x], [x, x]), ([x, a], [a, y]),
                        ([a], [flat[1:41]]), ([x, flat], [b, None]), ([x], [x.bfloat16().float()[:39]])):
        with pytest.raises(ValueError):
            moe.GradList(grads, outs)
    moe.GradList([x, x], [a, b])  # the same gradient twice is two summands
    moe.GradList([a, b], [a, b])
    moe.GradList([a, flat], None)
    norm, ws = torch.zeros(1, device="cuda"), torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    x.fill_(2.0)
    moe.clip_grad_norm(moe.GradList([x, x], [a, b]), 1.0, norm, ws)
    assert abs(norm.item() - (80 * 4) ** 0.5) < 1e-5 and torch.equal(a, b)


def test_bad_calls():
    lib, p = moe.load(), ctypes.c_void_p
    Grad = moe._Grad
    need = moe.clip_grad_norm_workspace_size(1)

    def call(n=1, scale=1.0, max_norm=1.0, eps=1e-6, norm=A, ws=A, ws_bytes=need, null=False, **kw):
        g = dict(grad=A, out=A, size=8, dtype=moe.F32, out_dtype=moe.F32)
        g.update(kw)
        arr = (Grad * 1)(Grad(g["grad"], g["out"], g["size"], g["dtype"], g["out_dtype"]))
        return lib.moe_clip_grad_norm(None if null else p(ctypes.addressof(arr)), n, scale,
                                      max_norm, eps, p(norm), p(ws), ws_bytes, None)

    inf, nan = float("inf"), float("nan")
    for kw in (dict(n=-1), dict(n=2 ** 20 + 1), dict(null=True), dict(size=-1),
               dict(size=2 ** 40 + 1), dict(dtype=2), dict(out_dtype=-1), dict(grad=None),
               dict(dtype=moe.BF16), dict(scale=0.0), dict(scale=inf), dict(scale=nan),
               dict(max_norm=0.0), dict(max_norm=nan), dict(max_norm=-1.0), dict(eps=-1.0),
               dict(eps=nan), dict(norm=None, out=None), dict(norm=None, n=0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(grad=A + 2), dict(out=A + 2), dict(norm=A + 1), dict(ws=A + 8)):
        assert call(**kw) == MISALIGNED, kw
    assert call(ws=None) == WORKSPACE and call(ws_bytes=need - 1) == WORKSPACE
    n = ctypes.c_size_t(0)
    assert lib.moe_clip_grad_norm_workspace_size(-1, ctypes.byref(n)) == INVALID
    assert lib.moe_clip_grad_norm_workspace_size(1, None) == INVALID
