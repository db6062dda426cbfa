"""Routing from scores (moe_route_scored) and its gradient against a plain 64-bit restatement.

The choice is defined on 64-bit keys, so the ids must be equal, near-ties among them.
Tolerances of the floats (u = 2^-24, the rounding of a float32 operation):
 - weights: two exponentials (2 units in the last place each), a sum of at most 16 terms and
   three roundings, under 32 u relative; without renormalisation the softmax's sum over the
   experts uses the hardware exponential, whose bound (2 + 1.17 |x|) 2^-23 averages to at most
   11 * 2^-21 with |x| under the entropy's ln 1024 = 7;
 - gradients: the same relative errors on each factor, on top of a difference of terms of the
   size of scale * max |dw|; bf16 gradients are rounded once more (2^-8).
"""

import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from mixture_experts_layer_04_gb300 import build as moe_build

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA, TIMEOUT, INTERNAL, MISALIGNED = range(8)
W_RTOL = 11 * 2.0 ** -21
G_RTOL = 64 * 2.0 ** -24


# ------------------------------------------------------------- the plain restatement ----

def scores(l, kind):
    """64-bit scores of one row; masked experts 0."""
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    ok = l > -np.inf
    s = np.zeros(l.shape)
    if ok.any():
        with np.errstate(over="ignore"):
            if kind == moe.SCORE_SIGMOID:
                s[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
            else:
                p = np.exp(l[ok] - l[ok].max())
                s[ok] = p / p.sum()
    return s, ok


def choose(c, l, bias):
    s, ok = scores(l, c.score)
    key = s + bias
    ok = ok & (bias > -np.inf)
    key = np.where(ok, key, -np.inf)
    per = c.E // c.groups
    if c.top_groups < c.groups:
        total = np.full(c.groups, -np.inf)
        for g in range(c.groups):
            k = np.sort(key[g * per:(g + 1) * per])[::-1][:c.group_rank]
            k = k[k > -np.inf]
            if k.size:
                total[g] = k.sum()
        keep = np.argsort(-total, kind="stable")[:c.top_groups]
        key = np.where(np.isin(np.arange(c.E) // per, keep), key, -np.inf)
    order = np.argsort(-key, kind="stable")[:c.K]
    order = order[key[order] > -np.inf]
    ids = np.full(c.K, -1, np.int64)
    ids[:order.size] = order
    w = np.zeros(c.K)
    kept = s[order]
    if order.size:
        if c.renormalise and kept.sum() == 0.0:  # scores under the smallest double: equal logits
            kept = np.ones(order.size)
        w[:order.size] = c.scale * kept / (kept.sum() if c.renormalise else 1.0)
    return ids, w


def reference(c, L, bias):
    b = np.zeros(c.E) if bias is None else np.asarray(bias, np.float64)
    rows = [choose(c, L[t], b) for t in range(c.T)]
    return np.array([r[0] for r in rows]).reshape(c.T, c.K), np.array([r[1] for r in rows]).reshape(c.T, c.K)


def weights_of(c, l, ids):
    """The weights as a function of one row's logits with the choice held."""
    s, _ = scores(l, c.score)
    kept = s[ids]
    return c.scale * kept / (kept.sum() if c.renormalise else 1.0)


def reference_grad(c, L, ids, dw):
    out = np.zeros((c.T, c.E))
    for t in range(c.T):
        s, ok = scores(L[t], c.score)
        live = np.array([i for i in range(c.K) if 0 <= ids[t, i] < c.E and ok[ids[t, i]]], int)
        if live.size == 0:
            continue
        at = ids[t, live]
        up = c.scale * dw[t, live]
        ds = np.zeros(c.E)
        if c.renormalise:
            S = s[at].sum()
            ds[at] = (up - (up * s[at]).sum() / S) / S
        else:
            ds[at] = up
        if c.score == moe.SCORE_SIGMOID:
            out[t] = ds * s * (1.0 - s)
        else:
            out[t] = s * (ds - (ds * s).sum())
    return out


# ------------------------------------------------------------------- host-side checks ----

@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def make(**kw):
    base = dict(T=4, E=64, K=4, groups=1, top_groups=1, group_rank=1, score=moe.SCORE_SIGMOID,
                renormalise=True, scale=1.0, dtype=moe.F32, logits_stride=0)
    base.update(kw)
    return moe.RouteConfig.make(**base)


A = ctypes.c_void_p(0x7000_0000_0000)  # never dereferenced: the calls below fail before a launch


@pytest.mark.parametrize("bad", [
    dict(K=0), dict(K=17), dict(K=9, E=8), dict(E=0), dict(E=1025, K=2), dict(T=-1),
    dict(groups=0), dict(groups=33, E=66), dict(groups=3), dict(top_groups=0),
    dict(groups=4, top_groups=5), dict(group_rank=0), dict(group_rank=3), dict(score=2),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(dtype=5), dict(logits_stride=63), dict(logits_stride=-64),
    dict(groups=16, top_groups=1, K=5), dict(T=1 << 30, K=4),
])
def test_invalid_configs_are_refused(lib, bad):
    c = make(**bad)
    assert lib.moe_route_scored(ctypes.byref(c), A, None, A, A, None) == INVALID
    assert lib.moe_route_scored_backward(ctypes.byref(c), A, A, A, A, None) == INVALID


def test_null_config_and_flag_values_are_refused(lib):
    assert lib.moe_route_scored(None, A, None, A, A, None) == INVALID
    c = make()
    c.renormalise = 2
    assert lib.moe_route_scored(ctypes.byref(c), A, None, A, A, None) == INVALID


def test_pointers_are_checked_before_a_launch(lib):
    c, off = make(), ctypes.c_void_p(0x7000_0000_0002)
    for i in (0, 2, 3):
        args = [A, None, A, A]
        args[i] = None
        assert lib.moe_route_scored(ctypes.byref(c), *args, None) == INVALID
        args[i] = off
        assert lib.moe_route_scored(ctypes.byref(c), *args, None) == MISALIGNED
    assert lib.moe_route_scored(ctypes.byref(c), A, off, A, A, None) == MISALIGNED
    for i in range(4):
        args = [A, A, A, A]
        args[i] = None
        assert lib.moe_route_scored_backward(ctypes.byref(c), *args, None) == INVALID
        args[i] = off
        assert lib.moe_route_scored_backward(ctypes.byref(c), *args, None) == MISALIGNED


def test_zero_tokens_and_injected_faults(lib):
    c = make(T=0)
    assert lib.moe_route_scored(ctypes.byref(c), None, None, None, None, None) == OK
    assert lib.moe_route_scored_backward(ctypes.byref(c), None, None, None, None, None) == OK
    for name in ("moe_route_scored", "moe_route_scored_backward"):
        moe.debug_set_fault(name, 1)
        fn = moe.route_scored if name == "moe_route_scored" else moe.route_scored_backward
        with pytest.raises(moe.MoEError):
            fn(c, None, None, None, None, stream=0)
        fn(c, None, None, None, None, stream=0)


def test_the_restated_gradient_agrees_with_differences():
    rng = np.random.default_rng(0)
    for score in (moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID):
        for renorm in (True, False):
            c = make(T=1, E=12, K=3, score=score, renormalise=renorm, scale=1.5)
            l = rng.normal(size=12)
            ids, _ = choose(c, l, np.zeros(12))
            dw = rng.normal(size=(1, 3))
            got = reference_grad(c, l[None], ids[None], dw)[0]
            for e in range(12):
                h = np.zeros(12)
                h[e] = 1e-6
                diff = (weights_of(c, l + h, ids) - weights_of(c, l - h, ids)) @ dw[0] / 2e-6
                assert abs(diff - got[e]) < 1e-8


# --------------------------------------------------------------------------- on a GPU ----

def run(c, logits, bias=None, stream=None):
    ids = torch.full((c.T, c.K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((c.T, c.K), float("nan"), device="cuda")
    moe.route_scored(c, logits, bias, ids, w, stream=stream)
    return ids, w


def check(c, logits, bias=None):
    ids, w = run(c, logits, bias)
    L = logits.double().cpu().numpy()[:, :c.E]
    rid, rw = reference(c, L, None if bias is None else bias.double().cpu().numpy())
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.double().cpu().numpy(), rw, rtol=W_RTOL, atol=1e-30)
    return ids, w


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


SHAPES = [  # T, E, K, groups, top_groups, rank
    (1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 1, 1), (5, 31, 7, 1, 1, 1), (33, 32, 8, 8, 3, 2),
    (17, 60, 4, 1, 1, 1), (9, 60, 6, 6, 2, 2), (64, 128, 8, 1, 1, 1), (40, 184, 5, 4, 2, 2),
    (130, 256, 8, 8, 4, 2), (11, 256, 16, 32, 9, 1), (21, 255, 10, 5, 3, 2),
    (10, 500, 16, 4, 1, 2), (7, 1024, 16, 32, 4, 2), (6, 1000, 3, 1, 1, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("shape", SHAPES)
def test_choice_and_weights(shape, score, dtype):
    T, E, K, G, TG, rank = shape
    g = gen(T * 1000 + E)
    logits = (torch.randn(T, E, generator=g, device="cuda") * 2).to(dtype)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    for renorm in (True, False):
        for b in (None, bias):
            c = moe.RouteConfig.make(T, E, K, G, TG, rank, score, renorm, 2.5,
                                     moe.BF16 if dtype == torch.bfloat16 else moe.F32)
            check(c, logits, b)


@pytest.mark.gpu
def test_many_tokens_have_the_64_bit_choice():
    # enough tokens that some choices are closer than float scores can tell
    g = gen(5)
    logits = torch.randn(6000, 256, generator=g, device="cuda")
    bias = torch.randn(256, generator=g, device="cuda") * 0.1
    for score in (moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID):
        c = moe.RouteConfig.make(6000, 256, 8, 8, 4, 2, score, True, 1.0)
        check(c, logits, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
def test_near_ties_are_decided_in_64_bits(score):
    # pairs of experts whose biased scores agree to about 1e-8: float keys cannot order them
    g = gen(6)
    T, E = 200, 64
    logits = torch.randn(T, E, generator=g, device="cuda")
    s = np.array([scores(row, score)[0] for row in logits.double().cpu().numpy()])
    b = np.zeros(E)
    b[1::2] = s[0, 0::2] - s[0, 1::2]  # token 0: every pair nearly tied
    bias = torch.tensor(b, dtype=torch.float32, device="cuda")
    logits[1:] = logits[0]             # and the same with logits a few units apart
    for t in range(1, T):
        logits[t, t % E] = torch.nextafter(logits[t, t % E],
                                           torch.tensor(9.0 if t % 2 else -9.0, device="cuda"))
    check(moe.RouteConfig.make(T, E, 8, 1, 1, 1, score), logits, bias)
    check(moe.RouteConfig.make(T, E, 8, 8, 4, 2, score), logits, bias)
    check(moe.RouteConfig.make(T, E, 8, 32, 16, 1, score), logits, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
def test_exact_ties_behind_a_near_tie(score):
    # many experts of equal logit and bias, and some just below them in 64 bits that float
    # keys cannot tell from them, at lower ids: the equal ones fill all places
    T, E = 40, 96
    logits = torch.zeros(T, E, device="cuda")
    bias = torch.full((E,), 0.25, device="cuda")
    below = torch.randperm(E, generator=torch.Generator().manual_seed(3))[:20]
    logits[:, below] = 1.0
    for t in range(T):  # a different number of experts out of the way in each row
        logits[t, 96 - t:] = -30.0
    s = np.array([scores(row, score)[0] for row in logits.double().cpu().numpy()])
    one, zero = int(below[0]), int([e for e in range(40) if e not in below.tolist()][0])
    gap = s[0, zero] + 0.25 - s[0, one]
    bias[below] = torch.tensor(np.nextafter(np.float32(gap), np.float32(-9.0)), device="cuda")
    for K in (1, 3, 8, 16):
        check(moe.RouteConfig.make(T, E, K, 1, 1, 1, score), logits, bias)
        check(moe.RouteConfig.make(T, E, K, 4, 3, 2, score), logits, bias)


@pytest.mark.gpu
def test_exact_ties_go_to_the_lower_id():
    for score in (moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID):
        for G, TG in ((1, 1), (8, 3)):
            c = moe.RouteConfig.make(5, 128, 8, G, TG, 2, score)
            logits = torch.zeros(5, 128, device="cuda")
            logits[1, 100:] = 1.0
            logits[2] = (torch.arange(128, device="cuda") % 4).float()
            logits[3] = -200.0
            logits[4] = 90.0
            check(c, logits)
            check(c, logits, torch.zeros(128, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
def test_masked_rows_infinities_and_nan(score):
    T, E = 12, 96
    logits = torch.randn(T, E, generator=gen(7), device="cuda")
    inf = float("inf")
    logits[0] = -inf                      # nothing available
    logits[1] = float("nan")
    logits[2, 3:] = -inf                  # fewer than K
    logits[3, ::2] = float("nan")
    logits[4, 5] = inf
    logits[5, [7, 50]] = inf              # +inf counts as the largest float: a tie
    logits[6] = torch.finfo(torch.float32).min  # the type's lowest value is not a mask
    logits[7, 1:] = torch.finfo(torch.float32).min
    logits[8, :32] = -inf                 # whole groups gone
    logits[9, 10:] = -inf
    bias = torch.randn(E, generator=gen(8), device="cuda") * 0.1
    bias[11] = -inf
    bias[12] = float("nan")
    for renorm in (True, False):
        for G, TG in ((1, 1), (3, 2), (12, 5)):
            c = moe.RouteConfig.make(T, E, 6, G, TG, 2, score, renorm)
            ids, w = check(c, logits)
            assert (ids[0] == -1).all() and (w[0] == 0).all()
            check(c, logits, bias)
            dl = torch.full((T, E), float("nan"), device="cuda")
            dw = torch.randn(T, 6, generator=gen(9), device="cuda")
            moe.route_scored_backward(c, logits, ids, dw, dl)
            assert torch.isfinite(dl).all()
            assert (dl[0] == 0).all() and (dl[3, ::2] == 0).all()


@pytest.mark.gpu
def test_strided_and_unaligned_rows():
    g = gen(10)
    wide = torch.randn(40, 259, generator=g, device="cuda")
    for off, stride in ((0, 259), (1, 259), (3, 259)):
        view = wide[:, off:off + 256]
        c = moe.RouteConfig.make(40, 256, 8, 8, 4, 2, moe.SCORE_SIGMOID, logits_stride=stride)
        check(c, view, torch.randn(256, generator=g, device="cuda") * 0.1)
    wb = torch.randn(40, 136, generator=g, device="cuda").bfloat16()
    c = moe.RouteConfig.make(40, 128, 8, dtype=moe.BF16, logits_stride=136)
    check(c, wb[:, 1:129])
    check(c, wb[:, :128])


def grad(c, logits, ids, dw, out=None):
    out = torch.full_like(logits, float("nan")) if out is None else out
    moe.route_scored_backward(c, logits, ids, dw, out)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradient(shape, renorm, score, dtype):
    T, E, K, G, TG, rank = shape
    g = gen(T * 1000 + E + 1)
    logits = (torch.randn(T, E, generator=g, device="cuda") * 2).to(dtype)
    dw = torch.randn(T, K, generator=g, device="cuda")
    c = moe.RouteConfig.make(T, E, K, G, TG, rank, score, renorm, 1.5,
                             moe.BF16 if dtype == torch.bfloat16 else moe.F32)
    ids, _ = run(c, logits)
    got = grad(c, logits, ids, dw).double().cpu().numpy()
    want = reference_grad(c, logits.double().cpu().numpy(), ids.cpu().numpy(),
                          dw.double().cpu().numpy())
    atol = G_RTOL * 1.5 * float(dw.abs().max())
    np.testing.assert_allclose(got, want, rtol=2.0 ** -8 if dtype == torch.bfloat16 else G_RTOL,
                               atol=atol)


@pytest.mark.gpu
def test_gradient_with_empty_slots_in_place_and_strided():
    g = gen(11)
    logits = torch.randn(20, 48, generator=g, device="cuda")
    logits[4] = float("-inf")
    logits[5, 2:] = float("-inf")
    dw = torch.randn(20, 6, generator=g, device="cuda")
    for score in (moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID):
        for renorm in (True, False):
            c = moe.RouteConfig.make(20, 48, 6, score=score, renormalise=renorm)
            ids, _ = run(c, logits)
            ids[7, 2] = 48          # outside: an empty slot, as -1
            ids[8] = -1
            want = reference_grad(c, logits.double().cpu().numpy(), ids.cpu().numpy(),
                                  dw.double().cpu().numpy())
            got = grad(c, logits, ids, dw)
            np.testing.assert_allclose(got.cpu().numpy(), want, rtol=G_RTOL,
                                       atol=G_RTOL * float(dw.abs().max()))
            same = logits.clone()
            assert torch.equal(grad(c, same, ids, dw, same), got)
            wide_in, wide_out = torch.zeros(20, 53, device="cuda"), torch.zeros(20, 53, device="cuda")
            wide_in[:, :48] = logits
            cs = moe.RouteConfig.make(20, 48, 6, score=score, renormalise=renorm, logits_stride=53)
            grad(cs, wide_in, ids, dw, wide_out)
            assert torch.equal(wide_out[:, :48], got) and (wide_out[:, 48:] == 0).all()


@pytest.mark.gpu
def test_saturated_and_tiny_scores_keep_finite_weights():
    for level in (-300.0, -90.0, -61.0, 100.0):
        logits = level + torch.randn(8, 64, generator=gen(12), device="cuda")
        c = moe.RouteConfig.make(8, 64, 4, score=moe.SCORE_SIGMOID)
        ids, w = check(c, logits)
        assert torch.allclose(w.sum(1), torch.ones(8, device="cuda"))
        dl = grad(c, logits, ids, torch.randn(8, 4, generator=gen(13), device="cuda"))
        assert torch.isfinite(dl).all()


@pytest.mark.gpu
def test_side_stream_and_graph_capture():
    g = gen(14)
    logits = torch.randn(50, 256, generator=g, device="cuda")
    bias = torch.randn(256, generator=g, device="cuda") * 0.1
    dw = torch.randn(50, 8, generator=g, device="cuda")
    c = moe.RouteConfig.make(50, 256, 8, 8, 4, 2, moe.SCORE_SIGMOID)
    ids0, w0 = check(c, logits, bias)
    dl0 = grad(c, logits, ids0, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids, w = torch.zeros_like(ids0), torch.zeros_like(w0)
    dl = torch.zeros_like(dl0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.route_scored(c, logits, bias, ids, w)
        moe.route_scored_backward(c, logits, ids, dw, dl)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, ids0) and torch.equal(w, w0) and torch.equal(dl, dl0)
    moe.sync_check()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    # more than 2^31 logits; the last rows equal a small call on them
    T, E, K, tail = 8_500_000, 256, 2, 64
    logits = torch.zeros(T, E, device="cuda")
    logits[-tail:] = torch.randn(tail, E, generator=gen(15), device="cuda")
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    c = moe.RouteConfig.make(T, E, K, score=moe.SCORE_SIGMOID)
    moe.route_scored(c, logits, None, ids, w)
    small = moe.RouteConfig.make(tail, E, K, score=moe.SCORE_SIGMOID)
    sid, sw = check(small, logits[-tail:])
    assert torch.equal(ids[-tail:], sid) and torch.equal(w[-tail:], sw)
    dw = torch.randn(T, K, generator=gen(16), device="cuda")
    moe.route_scored_backward(c, logits, ids, dw, logits)
    want = grad(small, torch.randn(tail, E, generator=gen(15), device="cuda"), sid,
                dw[-tail:].contiguous())
    assert torch.equal(logits[-tail:], want)
