"""The combine's gradient (moe_combine_backward) against the formula in 64 bits.

Tolerances: a dot of H float32 products summed in float32 by 32 to 256 partial sums of at most
H / 256 + 8 steps each is off by at most (H / 256 + 16) 2^-24 of the sum of the absolute
products; the rows are one product (2^-24) and one rounding (bf16 2^-8).
"""

import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from mixture_experts_layer_04_gb300 import build as moe_build

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA, TIMEOUT, INTERNAL, MISALIGNED = range(8)
A = ctypes.c_void_p(0x7000_0000_0000)


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def config(T=4, H=128, E=16, K=4, dtype=moe.BF16):
    return moe.MoEConfig.make(T=T, H=H, E=E, K=K, I=64, dtype=dtype)


def test_refusals(lib):
    c = config()
    call = lib.moe_combine_backward
    for i in (0, 2):
        args = [A] * 6
        args[i] = None
        assert call(ctypes.byref(c), *args, None) == INVALID
    assert call(ctypes.byref(c), A, A, A, A, None, None, None) == INVALID   # no output
    assert call(ctypes.byref(c), A, None, A, A, A, A, None) == INVALID      # d_w needs the rows
    assert call(ctypes.byref(c), A, A, A, None, A, A, None) == INVALID      # d_rows need w
    for i in range(6):
        args = [A] * 6
        args[i] = ctypes.c_void_p(0x7000_0000_0008)
        assert call(ctypes.byref(c), *args, None) == MISALIGNED
    bad = config(H=100)
    assert call(ctypes.byref(bad), A, A, A, A, A, A, None) == INVALID
    assert call(None, A, A, A, A, A, A, None) == INVALID
    empty = config(T=0)
    assert call(ctypes.byref(empty), None, None, None, None, None, None, None) == OK
    moe.debug_set_fault("moe_combine_backward", 1)
    with pytest.raises(moe.MoEError):
        moe.combine_backward(empty, None, None, None, None, None, None, stream=0)


def make(T, H, K, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dy = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    o = torch.randn(T * K, H, generator=g, device="cuda")
    w = torch.rand(T, K, generator=g, device="cuda")
    inv = torch.randperm(T * K, generator=g, device="cuda").to(torch.int32).view(T, K)
    return dy, o, inv, w


def reference(dy, o, inv, w):
    T, K = inv.shape
    at = inv.long().clamp(0, T * K - 1)
    live = (inv >= 0) & (inv < T * K)
    rows = o.double()[at]
    dw = torch.einsum("th,tkh->tk", dy.double(), rows) * live
    size = torch.einsum("th,tkh->tk", dy.double().abs(), rows.abs()) * live
    return dw, size, w.double()[:, :, None] * dy.double()[:, None, :]


def check(dy, o, inv, w, c):
    T, K = inv.shape
    H = dy.shape[1]
    d_o = torch.full((T * K, H), 77.0, dtype=dy.dtype, device="cuda")
    d_w = torch.full((T, K), float("nan"), device="cuda")
    moe.combine_backward(c, dy, o, inv, w, d_o, d_w)
    dw, size, rows = reference(dy, o, inv, w)
    assert ((d_w.double() - dw).abs() <= (H / 256 + 16) * 2.0 ** -24 * size + 1e-30).all()
    rtol = 2.0 ** -8 if dy.dtype == torch.bfloat16 else 2.0 ** -23
    touched = torch.zeros(T * K, dtype=torch.bool, device="cuda")
    for k in range(K):
        at = inv[:, k].long()
        ok = (at >= 0) & (at < T * K)
        got = d_o[at[ok]].double()
        want = rows[ok, k]
        assert ((got - want).abs() <= rtol * want.abs() + 1e-30).all()
        touched[at[ok]] = True
    assert (d_o[~touched] == 77.0).all()
    return d_o, d_w


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,K", [(1, 64, 1), (1, 7168, 8), (3, 192, 5), (16, 2048, 8),
                                   (100, 320, 10), (500, 256, 3), (1300, 128, 2), (700, 64, 16)])
def test_formula(T, H, K, dtype):
    c = config(T, H, 16, K, moe.BF16 if dtype == torch.bfloat16 else moe.F32)
    check(*make(T, H, K, dtype, seed=T + H), c)


@pytest.mark.gpu
def test_dropped_slots_bad_rows_and_single_outputs():
    dy, o, inv, w = make(40, 256, 4, torch.bfloat16, seed=3)
    inv[3] = -1
    inv[5, 1:] = -1
    inv[6, 2] = 160          # outside: as dropped
    inv[7, 0] = -(1 << 31)
    c = config(40, 256, 16, 4)
    d_o, d_w = check(dy, o, inv, w, c)
    assert (d_w[3] == 0).all() and d_w[6, 2] == 0
    only_w = torch.full_like(d_w, 5.0)
    moe.combine_backward(c, dy, o, inv, None, None, only_w)
    assert torch.equal(only_w, d_w)
    only_o = torch.full_like(d_o, 77.0)
    moe.combine_backward(c, dy, None, inv, w, only_o, None)
    assert torch.equal(only_o, d_o)


@pytest.mark.gpu
def test_untouched_values_do_not_leak():
    # NaN and infinities in rows no assignment maps to, or of another token, stay there
    dy, o, inv, w = make(20, 128, 4, torch.float32, seed=4)
    gone = inv[9].clone().long()
    inv[9] = -1
    o[gone] = float("nan")
    dy[9] = float("inf")
    d_o = torch.zeros_like(o)
    d_w = torch.zeros_like(w)
    moe.combine_backward(config(20, 128, 16, 4, moe.F32), dy, o, inv, w, d_o, d_w)
    assert torch.isfinite(d_o).all() and torch.isfinite(d_w).all() and (d_w[9] == 0).all()


@pytest.mark.gpu
def test_it_is_the_gradient_of_combine():
    # y from moe_combine in float32, differences of <dy, y> along random directions
    T, H, K = 12, 64, 3
    dy, o, inv, w = make(T, H, K, torch.float32, seed=5)
    c = config(T, H, 16, K, moe.F32)
    d_o, d_w = torch.zeros_like(o), torch.zeros_like(w)
    moe.combine_backward(c, dy, o, inv, w, d_o, d_w)

    def value(o_, w_):
        y = torch.empty(T, H, device="cuda")
        moe.combine(c, o_.contiguous(), inv, w_.contiguous(), None, y)
        return (y.double() * dy.double()).sum().item()

    g = torch.Generator(device="cuda").manual_seed(6)
    do, dw = torch.randn_like(o), torch.randn(T, K, generator=g, device="cuda")
    # y is linear in each argument: a whole step is exact up to float32 rounding of T*H sums
    scale = (dy.abs().double().sum() * 16).item()
    assert abs(value(o + do, w) - value(o, w) - (d_o.double() * do.double()).sum().item()) < 2.0 ** -20 * scale
    assert abs(value(o, w + dw) - value(o, w) - (d_w.double() * dw.double()).sum().item()) < 2.0 ** -20 * scale


@pytest.mark.gpu
def test_graph_capture_and_repeatability():
    dy, o, inv, w = make(64, 512, 8, torch.bfloat16, seed=8)
    c = config(64, 512, 16, 8)
    d_o, d_w = check(dy, o, inv, w, c)
    o2, w2 = torch.zeros_like(d_o), torch.zeros_like(d_w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.combine_backward(c, dy, o, inv, w, o2, w2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, d_o) and torch.equal(w2, d_w)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    # more than 2^31 values in the expert rows; the last tokens equal a small call on them
    T, H, K, tail = 38_000, 7168, 8, 16
    g = torch.Generator(device="cuda").manual_seed(9)
    dy = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    o = torch.zeros(T * K, H, device="cuda")
    o[-tail * K:] = torch.randn(tail * K, H, generator=g, device="cuda")
    w = torch.rand(T, K, generator=g, device="cuda")
    inv = torch.arange(T * K, dtype=torch.int32, device="cuda").view(T, K)
    d_o = torch.empty(T * K, H, dtype=torch.bfloat16, device="cuda")
    d_w = torch.empty(T, K, device="cuda")
    moe.combine_backward(config(T, H, 16, K), dy, o, inv, w, d_o, d_w)
    local = torch.arange(tail * K, dtype=torch.int32, device="cuda").view(tail, K)
    so, sw = check(dy[-tail:].contiguous(), o[-tail * K:].contiguous(), local,
                   w[-tail:].contiguous(), config(tail, H, 16, K))
    assert torch.equal(d_o[-tail * K:], so)
    assert (d_w[:-tail] == 0).all()
    assert torch.allclose(d_w[-tail:], sw, rtol=1e-4, atol=1e-2)
