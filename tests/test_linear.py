"""Linear layers (moe_linear, moe_linear_backward) against the formulas in 64 bits.

Tolerances, with S the sum of the absolute products of an output:
 - the tensor core truncates at each of its additions (one per 16 products), so bf16 operands
   accumulate at most (depth / 16 + 16) 2^-23 S; on the CUDA cores less;
 - float32 operands: six products of bf16 parts (what is left out is under 8 * 2^-24 S), added in
   the tensor core over at most 1024 values (6 * 64 additions), then rounded additions;
 - an activation multiplies that error by its largest slope (under 1.13) and adds a few units
   in the last place of float32 (2^-20 |z|);
 - each output is rounded once (bf16 2^-8 of its size, float32 2^-24);
 - bf16 gradients: dz is rounded to bf16 before the products, 2^-8 S.  Roundings are independent,
   so over a whole gradient their root mean square is under 2^-8 / sqrt(3) each.
"""

import ctypes
import math

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from mixture_experts_layer_04_gb300 import build as moe_build

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA, TIMEOUT, INTERNAL, MISALIGNED = range(8)
A = ctypes.c_void_p(0x7000_0000_0000)
ACTS = [moe.ACT_NONE, moe.ACT_RELU, moe.ACT_GELU, moe.ACT_GELU_TANH, moe.ACT_SILU]
BIG = ctypes.c_size_t(1 << 62)


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def config(rows=16, fin=64, fout=64, **kw):
    return moe.LinearConfig.make(rows, fin, fout, **kw)


# ------------------------------------------------------------------- host-side checks ----

@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=(1 << 30) + 1), dict(fin=0), dict(fout=0), dict(fin=(1 << 20) + 1),
    dict(fout=(1 << 20) + 1), dict(dtype=2), dict(dtype=moe.F32, out_dtype=moe.BF16),
    dict(out_dtype=9), dict(activation=5), dict(activation=-1), dict(x_stride=63),
    dict(w_stride=1), dict(residual_stride=63), dict(y_stride=63), dict(z_stride=-64),
    dict(dx_stride=63), dict(dw_stride=63), dict(x_stride=(1 << 31) + 8),
])
def test_invalid_configs_are_refused(lib, bad):
    c = config(**bad)
    n = ctypes.c_size_t(7)
    assert lib.moe_linear_workspace_size(ctypes.byref(c), ctypes.byref(n)) == INVALID
    assert n.value == 7
    assert lib.moe_linear(ctypes.byref(c), A, A, None, None, A, None, A, BIG, None) == INVALID
    assert lib.moe_linear_backward(ctypes.byref(c), A, A, A, A, A, A, A, A, BIG, None) == INVALID


def test_pointers_and_workspace_are_checked_before_a_launch(lib):
    c = config(activation=moe.ACT_SILU)
    off = ctypes.c_void_p(0x7000_0000_0002)
    odd = ctypes.c_void_p(0x7000_0000_0001)
    n = ctypes.c_size_t(0)
    assert lib.moe_linear_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.moe_linear_workspace_size(ctypes.byref(c), None) == INVALID
    assert lib.moe_linear_workspace_size(ctypes.byref(c), ctypes.byref(n)) == OK
    need = n.value
    fwd = lambda *a, ws=A, nb=BIG: lib.moe_linear(ctypes.byref(c), *a, ws, nb, None)
    assert fwd(None, A, None, None, A, None) == INVALID
    assert fwd(A, None, None, None, A, None) == INVALID
    assert fwd(A, A, None, None, None, None) == INVALID
    assert fwd(off, A, None, None, A, None) == MISALIGNED   # read in place: 16 bytes
    assert fwd(A, off, None, None, A, None) == MISALIGNED
    assert fwd(A, A, off, None, A, None) == MISALIGNED
    for i in (3, 4, 5):
        args = [A, A, None, A, A, A]
        args[i] = odd
        assert fwd(*args) == MISALIGNED
    assert fwd(A, A, None, None, A, None, ws=None) == WORKSPACE
    assert fwd(A, A, None, None, A, None, nb=ctypes.c_size_t(need - 1)) == WORKSPACE
    assert fwd(A, A, None, None, A, None, ws=ctypes.c_void_p(0x7000_0000_0008)) == MISALIGNED
    bwd = lambda *a, ws=A, nb=BIG: lib.moe_linear_backward(ctypes.byref(c), *a, ws, nb, None)
    assert bwd(None, A, A, A, A, A, A) == INVALID
    assert bwd(A, A, A, None, A, A, A) == INVALID           # the activation needs z
    assert bwd(A, None, A, A, A, A, A) == INVALID           # dw needs x
    assert bwd(A, A, None, A, A, A, A) == INVALID           # dx needs w
    assert bwd(A, A, A, A, None, None, None) == INVALID     # no output
    assert bwd(off, A, A, A, A, A, A) == MISALIGNED
    assert bwd(A, A, A, odd, A, A, A) == MISALIGNED
    assert bwd(A, A, A, A, odd, A, A) == MISALIGNED
    assert bwd(A, A, A, A, A, A, off) == MISALIGNED
    assert bwd(A, A, A, A, A, A, A, nb=ctypes.c_size_t(need - 1)) == WORKSPACE


def test_strides_off_16_bytes_need_only_the_alignment_of_an_element(lib):
    c = config(x_stride=65)
    odd = ctypes.c_void_p(0x7000_0000_0001)
    assert lib.moe_linear(ctypes.byref(c), odd, A, None, None, A, None, A, BIG, None) == MISALIGNED
    plain, strided = config(), c
    assert moe.linear_workspace_size(strided) > moe.linear_workspace_size(plain)


def test_no_rows_and_injected_faults(lib):
    c = config(rows=0)
    assert lib.moe_linear(ctypes.byref(c), None, None, None, None, None, None, None, 0, None) == OK
    assert lib.moe_linear_backward(ctypes.byref(c), None, None, None, None, A, None, None, None, 0,
                                   None) == OK
    for name in ("moe_linear", "moe_linear_backward", "moe_linear_workspace_size"):
        moe.debug_set_fault(name, 1)
        with pytest.raises(moe.MoEError):
            if name == "moe_linear":
                moe.linear(c, None, None, None, None, None, stream=0)
            elif name == "moe_linear_backward":
                moe.linear_backward(c, None, None, None, None, None, None, None, stream=0)
            else:
                moe.linear_workspace_size(c)


# ----------------------------------------------------------------- formulas in 64 bits ----

def act(a, z):
    if a == moe.ACT_RELU:
        return z.clamp(min=0)
    if a == moe.ACT_GELU:
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if a == moe.ACT_GELU_TANH:
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if a == moe.ACT_SILU:
        return z * torch.sigmoid(z)
    return z


def slope(a, z):
    z = z.detach().clone().requires_grad_(True)
    act(a, z).sum().backward() if a != moe.ACT_NONE else z.sum().backward()
    return z.grad


def product_error(depth, size, f32, out_f32=False):
    if f32:
        adds = 6 * math.ceil(min(depth, 1024) / 16) + depth / 1024 + 16
    elif out_f32:
        adds = math.ceil(min(depth, 1024) / 16) + depth / 1024 + 16
    else:
        adds = depth / 16 + 16
    return adds * 2.0 ** -23 * size


def make(rows, fin, fout, dtype, seed, pad=0, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    wide = torch.full((rows, fin + pad), float("nan"), device="cuda")
    wide[:, off:off + fin] = r(rows, fin)
    x = wide.to(dtype)[:, off:off + fin]
    w = (r(fout, fin) * fin ** -0.5).to(dtype)
    return x, w, r(fout), r(rows, fout).to(dtype), g


def workspace(c):
    return torch.full((moe.linear_workspace_size(c),), 0xFF, dtype=torch.uint8, device="cuda")


def forward(rows, fin, fout, dtype, a, bias=True, residual=True, keep=True, out_f32=False, pad=0,
            off=0, seed=0):
    x, w, b, res, _ = make(rows, fin, fout, dtype, seed, pad, off)
    code = moe.BF16 if dtype == torch.bfloat16 else moe.F32
    c = config(rows, fin, fout, dtype=code, out_dtype=moe.F32 if out_f32 else code, activation=a,
               x_stride=fin + pad)
    y = torch.full((rows, fout), float("nan"), dtype=torch.float32 if out_f32 else dtype,
                   device="cuda")
    z = torch.full((rows, fout), float("nan"), dtype=dtype, device="cuda") if keep else None
    moe.linear(c, x, w, b if bias else None, res if residual else None, y, z, workspace(c))
    moe.sync_check()
    zr = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    if bias:
        zr = zr + b.double()
    yr = act(a, zr)
    if residual:
        yr = yr + res.double()
    f32 = dtype == torch.float32
    err = product_error(fin, size, f32, out_f32) + 2.0 ** -22 * (zr.abs() + 4)
    step = 2.0 ** -24 if (f32 or out_f32) else 2.0 ** -8
    assert ((y.double() - yr).abs() <= 1.13 * err + 2.0 ** -20 * zr.abs() + step * yr.abs() * 1.01).all()
    if keep:
        zstep = 2.0 ** -24 if f32 else 2.0 ** -8
        assert ((z.double() - zr).abs() <= err + zstep * zr.abs() * 1.01).all()
    if f32 or out_f32:
        assert (y.double() - yr).norm() <= 1e-5 * yr.norm()
    return c, x, w, b, res, y, z


SHAPES = [  # rows, in, out
    (1, 1, 1), (1, 4096, 513), (2, 100, 64), (3, 257, 33), (5, 64, 1), (8, 1000, 260),
    (9, 64, 64), (12, 7, 5), (16, 512, 300), (17, 40, 1030), (33, 2048, 256), (64, 4096, 200),
    (65, 72, 136), (100, 1, 100), (128, 1024, 128), (130, 65, 129), (200, 3000, 16),
    (300, 520, 2), (257, 1101, 511),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype):
    forward(*shape, dtype, moe.ACT_SILU, seed=shape[0])
    forward(*shape, dtype, moe.ACT_NONE, bias=False, residual=False, keep=False, seed=shape[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("a", ACTS)
def test_activations(a, dtype):
    forward(4, 130, 70, dtype, a)
    forward(70, 130, 70, dtype, a)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,fin,fout", [(4096, 200, 2048), (3999, 64, 2050), (2500, 1032, 2500)])
def test_forward_on_cta_pairs(rows, fin, fout):
    forward(rows, fin, fout, torch.bfloat16, moe.ACT_GELU_TANH)
    forward(rows, fin, fout, torch.bfloat16, moe.ACT_NONE, bias=False, residual=False, keep=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,fin,fout", [(185, 1024, 5440), (130, 200, 5437), (192, 72, 5440)])
def test_more_rows_than_a_tile_through_many_features(rows, fin, fout, dtype):
    forward(rows, fin, fout, dtype, moe.ACT_GELU, seed=rows)
    forward(rows, fin, fout, dtype, moe.ACT_NONE, bias=False, residual=False, keep=False, pad=5,
            off=3)
    if dtype == torch.bfloat16:
        forward(rows, fin, fout, dtype, moe.ACT_SILU, out_f32=True)


@pytest.mark.gpu
@pytest.mark.parametrize("pad,off", [(16, 16), (16, 8), (8, 0), (8, 8), (5, 3), (2, 1)])
@pytest.mark.parametrize("rows,fout", [(2560, 2048), (2500, 2500)])
def test_outputs_at_each_alignment_on_cta_pairs(rows, fout, pad, off):
    # 32-, 16- and 2-byte aligned rows are written in different ways; what lies beside them stays
    fin = 64
    x, w, b, res, _ = make(rows, fin, fout, torch.bfloat16, pad + off)
    wide = lambda: torch.full((rows, fout + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    y, z, r = wide(), wide(), wide()
    cut = lambda t: t[:, off:off + fout]
    cut(r).copy_(res)
    c = config(rows, fin, fout, activation=moe.ACT_SILU, y_stride=fout + pad, z_stride=fout + pad,
               residual_stride=fout + pad)
    moe.linear(c, x, w, b, cut(r), cut(y), cut(z), workspace(c))
    moe.sync_check()
    for t in (y, z):
        assert (t[:, :off] == 7).all() and (t[:, off + fout:] == 7).all()
    zr = x.double() @ w.double().t() + b.double()
    yr = act(moe.ACT_SILU, zr) + res.double()
    err = (product_error(fin, x.double().abs() @ w.double().abs().t(), False) +
           2.0 ** -22 * (zr.abs() + 4))
    assert ((cut(z).double() - zr).abs() <= err + 2.0 ** -8 * zr.abs() * 1.01).all()
    assert ((cut(y).double() - yr).abs() <=
            1.13 * err + 2.0 ** -20 * zr.abs() + 2.0 ** -8 * yr.abs() * 1.01).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (5, 0), (5, 3), (1, 1)])
def test_column_slices_do_not_read_their_neighbours(pad, off, dtype):
    # everything beside the slice is NaN
    for rows in (3, 20, 150):
        forward(rows, 96, 80, dtype, moe.ACT_RELU, pad=pad, off=off)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 7, 40, 1000])
def test_float32_results_of_bf16_operands(rows):
    forward(rows, 7168, 256, torch.bfloat16, moe.ACT_NONE, residual=False, keep=False, out_f32=True)
    forward(rows, 300, 60, torch.bfloat16, moe.ACT_SILU, out_f32=True)


@pytest.mark.gpu
def test_long_float32_sums_stay_float32():
    forward(150, 14336, 64, torch.float32, moe.ACT_NONE, residual=False, keep=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [2, 24, 200])
def test_residual_in_place_and_strided_outputs(rows, dtype):
    fin, fout = 128, 90
    c0, x, w, b, res, y0, z0 = forward(rows, fin, fout, dtype, moe.ACT_GELU)
    y = res.clone()
    moe.linear(c0, x, w, b, y, y, None, workspace(c0))
    assert torch.equal(y, y0)
    code = c0.dtype
    c = config(rows, fin, fout, dtype=code, activation=moe.ACT_GELU, residual_stride=101,
               y_stride=97, z_stride=95)
    rw = torch.zeros(rows, 101, dtype=dtype, device="cuda")
    rw[:, :fout] = res
    yw = torch.full((rows, 97), 7.0, dtype=dtype, device="cuda")
    zw = torch.full((rows, 95), 7.0, dtype=dtype, device="cuda")
    moe.linear(c, x, w, b, rw, yw, zw, workspace(c))
    assert torch.equal(yw[:, :fout], y0) and (yw[:, fout:] == 7).all()
    assert torch.equal(zw[:, :fout], z0) and (zw[:, fout:] == 7).all()


# ---------------------------------------------------------------------------- gradients ----

def backward(rows, fin, fout, dtype, a, bias=True, out_f32=False, pad=0, off=0, seed=0):
    x, w, _, z, g = make(rows, fin, fout, dtype, seed, pad, off)
    f32 = dtype == torch.float32
    code = moe.F32 if f32 else moe.BF16
    ydt = torch.float32 if out_f32 else dtype
    dy = torch.randn(rows, fout, generator=g, device="cuda").to(ydt)
    c = config(rows, fin, fout, dtype=code, out_dtype=moe.F32 if out_f32 else code, activation=a,
               x_stride=fin + pad)
    dx = torch.full((rows, fin), float("nan"), dtype=dtype, device="cuda")
    dw = torch.full((fout, fin), float("nan"), dtype=dtype, device="cuda")
    db = torch.full((fout,), float("nan"), device="cuda") if bias else None
    zz = z if a != moe.ACT_NONE else None
    moe.linear_backward(c, dy, x, w, zz, dx, dw, db, workspace(c))
    moe.sync_check()
    dz = dy.double() * slope(a, z.double())
    ad, xd, wd = dz.abs(), x.double(), w.double()
    rounding = 0.0 if f32 else 2.0 ** -8
    step = 2.0 ** -24 if f32 else 2.0 ** -8
    for got, want, size, depth in ((dx, dz @ wd, ad @ wd.abs(), fout),
                                   (dw, dz.t() @ xd, ad.t() @ xd.abs(), rows)):
        err = product_error(depth, size, f32) + (rounding + 2.0 ** -20) * size
        assert ((got.double() - want).abs() <= err + step * want.abs() * 1.01 + 1e-30).all()
        if want.norm() > 0 and got.numel() > 64:
            assert (got.double() - want).norm() <= (1e-5 if f32 else 2.0 ** -8) * want.norm()
    if bias:
        size = ad.sum(0)
        assert ((db.double() - dz.sum(0)).abs() <= (rows / 8 + 32) * 2.0 ** -24 * size +
                2.0 ** -20 * size + 1e-30).all()
    return c, dy, x, w, zz, dx, dw, db


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype):
    backward(*shape, dtype, moe.ACT_SILU, seed=shape[0])
    backward(*shape, dtype, moe.ACT_NONE, bias=False, seed=shape[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("a", ACTS)
def test_backward_activations(a, dtype):
    backward(70, 130, 70, dtype, a)


@pytest.mark.gpu
def test_backward_on_cta_pairs():
    backward(3999, 2050, 2048, torch.bfloat16, moe.ACT_GELU)
    backward(4096, 2048, 2056, torch.bfloat16, moe.ACT_NONE)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,fin,fout", [(70, 192, 5312), (60, 64, 8001), (333, 190, 5312),
                                           (100, 8000, 130)])
def test_backward_of_long_and_short_reductions(rows, fin, fout, dtype):
    # one gradient has few tiles and a long reduction, the other many tiles and a short one
    backward(rows, fin, fout, dtype, moe.ACT_GELU, seed=fout)
    backward(rows, fin, fout, dtype, moe.ACT_NONE, pad=5, off=3)


@pytest.mark.gpu
@pytest.mark.parametrize("pad,off", [(8, 8), (5, 3)])
def test_backward_of_column_slices(pad, off):
    for dtype in (torch.bfloat16, torch.float32):
        backward(40, 96, 72, dtype, moe.ACT_RELU, pad=pad, off=off)


@pytest.mark.gpu
def test_backward_of_float32_results():
    backward(100, 256, 60, torch.bfloat16, moe.ACT_NONE, out_f32=True)
    backward(37, 100, 256, torch.bfloat16, moe.ACT_SILU, out_f32=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_single_gradients_equal_the_joint_ones(dtype):
    c, dy, x, w, z, dx, dw, db = backward(150, 200, 120, dtype, moe.ACT_GELU)
    for only in range(3):
        outs = [torch.full_like(t, 3.0) for t in (dx, dw, db)]
        args = [o if i == only else None for i, o in enumerate(outs)]
        moe.linear_backward(c, dy, x if only == 1 else None, w if only == 0 else None, z, *args,
                            workspace(c))
        assert torch.equal(outs[only], (dx, dw, db)[only])


@pytest.mark.gpu
def test_backward_without_rows_zeroes_the_weight_gradients():
    c = config(0, 24, 10, dw_stride=30)
    dw = torch.full((10, 30), 5.0, dtype=torch.bfloat16, device="cuda")
    db = torch.full((10,), 5.0, device="cuda")
    moe.linear_backward(c, None, None, None, None, None, dw, db, None)
    assert (dw[:, :24] == 0).all() and (dw[:, 24:] == 5).all() and (db == 0).all()


@pytest.mark.gpu
def test_gradients_agree_with_differences():
    # float32, a direction at a time: the value is <dy, y>
    rows, fin, fout = 12, 20, 9
    for a in ACTS:
        x, w, b, _, g = make(rows, fin, fout, torch.float32, 3)
        c = config(rows, fin, fout, dtype=moe.F32, activation=a)
        dy = torch.randn(rows, fout, generator=g, device="cuda")
        y, z = torch.empty(rows, fout, device="cuda"), torch.empty(rows, fout, device="cuda")
        x, w = x.contiguous(), w.contiguous()
        moe.linear(c, x, w, b, None, y, z, workspace(c))
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        moe.linear_backward(c, dy, x, w, z, dx, dw, db, workspace(c))

        def value(x_, w_, b_):
            return (act(a, x_ @ w_.t() + b_) * dy.double()).sum().item()

        h = 1e-6
        for i, grad in enumerate((dx, dw, db)):
            base = [x.double(), w.double(), b.double()]
            d = torch.randn(grad.shape, generator=g, device="cuda").double()
            up, down = list(base), list(base)
            up[i] = base[i] + h * d
            down[i] = base[i] - h * d
            diff = (value(*up) - value(*down)) / (2 * h)
            assert abs(diff - (grad.double() * d).sum().item()) <= 1e-4 * (1 + abs(diff))


@pytest.mark.gpu
def test_calls_repeat_bit_for_bit_and_in_a_graph():
    rows, fin, fout = 48, 1024, 160
    c, x, w, b, res, y0, z0 = forward(rows, fin, fout, torch.bfloat16, moe.ACT_SILU)
    dy = torch.randn(rows, fout, device="cuda").bfloat16()
    ws = workspace(c)
    grads0 = [torch.empty_like(x.contiguous()), torch.empty_like(w), torch.empty_like(b)]
    moe.linear_backward(c, dy, x, w, z0, *grads0, ws)
    y, z = torch.zeros_like(y0), torch.zeros_like(z0)
    grads = [torch.zeros_like(t) for t in grads0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.linear(c, x, w, b, res, y, z, ws)
        moe.linear_backward(c, dy, x, w, z, *grads, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(z, z0)
    assert all(torch.equal(p, q) for p, q in zip(grads, grads0))
    moe.sync_check()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    # more than 2^31 elements in y, z and dy; the last rows are compared
    rows, fin, fout, tail = 270_000, 64, 8192, 300
    x, w, b, _, g = make(rows, fin, fout, torch.bfloat16, 5)
    x = x.contiguous()
    c = config(rows, fin, fout, activation=moe.ACT_SILU)
    y = torch.empty(rows, fout, dtype=torch.bfloat16, device="cuda")
    z = torch.empty_like(y)
    ws = torch.empty(moe.linear_workspace_size(c), dtype=torch.uint8, device="cuda")
    moe.linear(c, x, w, b, None, y, z, ws)
    zr = x[-tail:].double() @ w.double().t() + b.double()
    assert ((z[-tail:].double() - zr).abs() <= 2.0 ** -8 * zr.abs() * 1.01 + 1e-4).all()
    assert ((y[-tail:].double() - act(moe.ACT_SILU, zr)).abs()
            <= 2.0 ** -8 * zr.abs() * 1.01 + 1e-4).all()
    # dy is zero but for the last rows, so every gradient is theirs
    y.zero_()
    y[-tail:] = torch.randn(tail, fout, generator=g, device="cuda").bfloat16()
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    moe.linear_backward(c, y, x, w, z, dx, dw, db, ws)
    moe.sync_check()
    dz = y[-tail:].double() * slope(moe.ACT_SILU, z[-tail:].double())
    assert (dx[:-tail] == 0).all()
    for got, want in ((dx[-tail:], dz @ w.double()), (dw, dz.t() @ x[-tail:].double())):
        assert (got.double() - want).norm() <= 2.0 ** -8 * want.norm()
    assert (db.double() - dz.sum(0)).norm() <= 2.0 ** -18 * dz.abs().sum(0).norm()
