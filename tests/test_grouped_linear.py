"""Products grouped by expert and their gradients against 64-bit torch.

Tolerances.  S is the sum of the products' absolute values.  A bf16 result is rounded once: 2^-8 of
itself.  The tensor core adds 16 products at a time and truncates: at most 2^-22 of S a step, and a
float32 addition per chunk of 64 values or more of at most 2^-24 of S: ACC(n) = (n / 16 + n / 128 +
2) 2^-22.  Float32 operands are three bf16 parts (2^-24 of each value left, twice) and six products
per value, added in as many steps: 6 ACC(n) + 2^-22.  dz is rounded to bf16 once (2^-8 of itself,
and so of S of the products that take it; 2^-17 where dx is float32), SwiGLU's fast exponential is
good to 2e-5.  What a sum of independent roundings comes to is checked in L2: a product p_i whose factor is rounded is off by e_i p_i, with
e_i at most 2^-8 and 2^-8 / sqrt(3) in the root mean square, so sum e_i p_i has the root mean square
2^-8 / sqrt(3) sqrt(sum p_i^2) (not a share of the sum itself, whose terms may cancel), and the
result's own rounding adds 2^-8 / sqrt(3) of it; twice that is the bound.
"""

import ctypes

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe

OK, INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED = 0, 1, 2, 3, 7
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {BF16: moe.BF16, F32: moe.F32}
HALF = 2.0 ** -8
L2 = 2 * HALF / 3 ** 0.5


def acc(n, dtype):
    one = (n / 16 + n / 128 + 2) * 2.0 ** -22
    return 6 * one + 2.0 ** -22 if dtype == F32 else one


def step(dtype):
    return HALF if dtype == BF16 else 2.0 ** -24


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def sliced(g, rows, cols, pad, dtype, std=1.0):
    return randn(g, rows, cols + pad, dtype=dtype, std=std)[:, :cols]


class Case:
    """Operands of one set of group sizes; rows of no group are NaN in every input."""

    def __init__(self, sizes, fin, fout, act, dtype=BF16, out=None, dx=None, pad=0, tail=0, head=0,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes, self.fin, self.fout, self.act, self.dtype = sizes, fin, fout, act, dtype
        self.out, self.dxt = out or dtype, dx or dtype
        self.N = fout * (2 if act else 1)
        self.G, self.head = len(sizes), head
        used = sum(sizes)
        self.rows = rows = head + used + tail
        self.bounds = [head]
        for n in sizes:
            self.bounds.append(self.bounds[-1] + n)
        self.offsets = torch.tensor(self.bounds, dtype=torch.int32, device="cuda")
        self.x = sliced(g, rows, fin, pad, dtype)
        self.w = sliced(g, self.G * self.N, fin, pad, dtype, fin ** -0.5)
        self.dy = sliced(g, rows, fout, pad, dtype)
        self.z = sliced(g, rows, self.N, pad, dtype)
        for t in (self.x, self.dy, self.z):
            t[:head] = float("nan")
            t[head + used:] = float("nan")
        for e, n in enumerate(sizes):
            if n == 0:
                self.w[e * self.N:(e + 1) * self.N] = float("nan")
        self.pad = pad
        self.cfg = moe.GroupedConfig.make(
            rows, self.G, fin, fout, TYPES[dtype], TYPES[self.out], TYPES[self.dxt],
            moe.ACT_SWIGLU if act else moe.ACT_NONE, x_stride=fin + pad, w_stride=fin + pad,
            y_stride=fout + pad, z_stride=self.N + pad, dx_stride=fin + pad, dw_stride=fin + pad)
        self.ws = torch.full((moe.grouped_linear_workspace_size(self.cfg),), 255,
                             dtype=torch.uint8, device="cuda")

    def buffer(self, rows, cols, dtype):
        return torch.full((rows, cols + self.pad), 7.0, dtype=dtype, device="cuda")

    def forward(self, keep=True, **kw):
        y = self.buffer(self.rows, self.fout, self.out)
        z = self.buffer(self.rows, self.N, self.dtype) if self.act and keep else None
        moe.grouped_linear(self.cfg, self.x, self.offsets, self.w, y, z, self.ws, **kw)
        return y, z

    def backward(self, want_dx=True, want_dw=True, **kw):
        dx = self.buffer(self.rows, self.fin, self.dxt) if want_dx else None
        dw = self.buffer(self.G * self.N, self.fin, self.dtype) if want_dw else None
        moe.grouped_linear_backward(self.cfg, self.dy, self.x, self.offsets, self.w,
                                    self.z if self.act else None, dx, dw, self.ws, **kw)
        return dx, dw

    def groups(self):
        for e in range(self.G):
            a, b = self.bounds[e], self.bounds[e + 1]
            if a < b:
                yield e, slice(a, b), self.w[e * self.N:(e + 1) * self.N].double()

    def unowned(self, t, cols):
        """What no group and no column owns stays as it was."""
        assert (t[:self.head] == 7).all() and (t[self.bounds[-1]:] == 7).all()
        assert (t[:, cols:] == 7).all()

    def check_forward(self, y, z):
        F = self.fout
        self.unowned(y, F)
        if z is not None:
            self.unowned(z, self.N)
        for e, at, w in self.groups():
            x = self.x[at].double()
            ref, S = x @ w.t(), x.abs() @ w.abs().t()
            dz = S * acc(self.fin, self.dtype)
            if z is not None:
                assert_close(z[at, :self.N], ref, dz + step(self.dtype) * ref.abs())
            if self.act:
                g, u = ref[:, :F], ref[:, F:]
                value = torch.nn.functional.silu(g)
                fast = 2e-5 if self.dtype == BF16 else 2.0 ** -21
                tol = (1.1 * dz[:, :F] * (u.abs() + dz[:, F:]) + value.abs() * dz[:, F:]
                       + fast * (value * u).abs())
                ref = value * u
            else:
                tol = dz
            assert_close(y[at, :F], ref, tol + step(self.out) * ref.abs() + 1e-37)

    def dz(self, at):
        dy = self.dy[at].double()
        if not self.act:
            return dy
        g, u = self.z[at, :self.fout].double(), self.z[at, self.fout:self.N].double()
        s = torch.sigmoid(g)
        return torch.cat([dy * u * (s + g * s * (1 - s)), dy * g * s], dim=1)

    def check_backward(self, dx, dw):
        off = (HALF + 4e-5 if self.dtype == BF16 else 2.0 ** -21) if self.act else 0.0
        if dx is not None:
            self.unowned(dx, self.fin)
        if dw is not None:
            assert (dw[:, self.fin:] == 7).all()
        seen = set()
        for e, at, w in self.groups():
            seen.add(e)
            d, x = self.dz(at), self.x[at].double()
            two = self.dtype == BF16 and self.dxt == F32 and self.act  # dz in two parts for dx
            for got, a, b, t, rounded in (
                    (dx[at] if dx is not None else None, d, w, self.dxt,
                     2.0 ** -17 + 4e-5 if two else off),
                    (dw[e * self.N:(e + 1) * self.N] if dw is not None else None, d.t(), x,
                     self.dtype, off)):
                if got is not None:
                    got, ref, S, n = got[:, :self.fin], a @ b, a.abs() @ b.abs(), a.shape[1]
                    assert_close(got, ref, S * (acc(n, self.dtype) + rounded) * (1 + HALF)
                                 + step(t) * ref.abs() + 1e-37)
                    if self.dtype == BF16:
                        size = ref.norm() + (a ** 2 @ b ** 2).sum().sqrt()
                        assert ((got.double() - ref).norm() / size).item() < L2
        if dw is not None:
            for e in range(self.G):
                if e not in seen:
                    assert (dw[e * self.N:(e + 1) * self.N, :self.fin] == 0).all()


def assert_close(got, ref, tol):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), got.double()[bad][:4].tolist(), ref[bad][:4].tolist(),
                           tol[bad][:4].tolist())


# few rows a group (the weights on the side of 128) and many (CTA pairs), ragged and empty groups,
# one group, many groups
SIZES = [
    [1], [0, 1, 0], [3, 0, 1, 7, 32, 33, 31], [5] * 40, [0] * 9 + [70, 0, 64, 63, 1],
    [300], [256, 1, 0, 257, 511, 64], [1000, 0, 17, 2300],
]


@pytest.mark.gpu
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("fin,fout", [(64, 64), (200, 136), (1024, 512)])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_bf16(sizes, fin, fout, act):
    c = Case(sizes, fin, fout, act, tail=5, seed=fin)
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())
    moe.sync_check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes", [[i % 3 for i in range(1024)], [0] * 1023 + [900],
                                   [200] + [0] * 500 + [3] * 200, [65 + i for i in range(300)]],
                         ids=["1024 groups", "the last", "few of 701", "300 groups"])
def test_many_groups(sizes, dtype):
    c = Case(sizes, 72, 64, True, dtype=dtype, tail=7, seed=12)
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())
    moe.sync_check()


@pytest.mark.gpu
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("sizes", [[4, 0, 30], [70, 1, 0, 200], [600, 300]], ids=str)
def test_float32_results(sizes, act):
    c = Case(sizes, 320, 192, act, out=F32, dx=F32, tail=2, seed=1)
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("fin,fout,pad", [(1, 1, 0), (7, 5, 0), (65, 33, 1), (333, 201, 3),
                                          (130, 70, 8), (129, 127, 0)])
@pytest.mark.parametrize("sizes", [[2, 0, 40], [129, 3, 0, 260]], ids=str)
def test_odd_sizes_and_strides(sizes, fin, fout, pad, act, dtype):
    c = Case(sizes, fin, fout, act, dtype=dtype, pad=pad, tail=3, head=4, seed=2)
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())
    moe.sync_check()


@pytest.mark.gpu
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("sizes", [[1, 0, 5], [64, 65, 0, 257]], ids=str)
def test_float32(sizes, act):
    c = Case(sizes, 512, 256, act, dtype=F32, tail=1, seed=3)
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_group_of_infinities_stays_in_its_rows(dtype):
    c = Case([100, 33, 77, 200], 192, 128, False, dtype=dtype, seed=4)
    for t in (c.x, c.dy):
        t[100:133] = float("inf")
        t[110] = float("nan")
    y, _ = c.forward()
    dx, dw = c.backward()
    for e in (0, 2, 3):
        at = slice(c.bounds[e], c.bounds[e + 1])
        w = c.w[e * c.N:(e + 1) * c.N].double()
        x, dy = c.x[at].double(), c.dy[at].double()
        for got, ref in ((y[at], x @ w.t()), (dx[at], dy @ w),
                         (dw[e * c.N:(e + 1) * c.N], dy.t() @ x)):
            assert ((got.double() - ref).norm() / ref.norm()).item() < HALF
    assert not torch.isfinite(y[100:133]).any()
    assert not torch.isfinite(dw[c.N:2 * c.N]).any()


@pytest.mark.gpu
def test_a_long_reduction_keeps_its_sums():
    # positive values: a truncating accumulator would fall short by 6e-9 of the sum per value
    n = 40000
    c = Case([n, 10], 64, 64, False, seed=5)
    c.x.abs_()
    c.dy.abs_()
    _, dw = c.backward(want_dx=False)
    ref = c.dy[:n].double().t() @ c.x[:n].double()
    assert ((dw[:64].double() / ref - 1).abs() <= HALF + 2e-4).all()


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[3, 0, 9], [300, 40, 0, 90]], ids=str)
def test_gradients_alone_and_repeated(sizes):
    c = Case(sizes, 256, 128, True, tail=2, seed=6)
    dx, dw = c.backward()
    for _ in range(3):
        assert torch.equal(c.backward(want_dw=False)[0], dx)
        assert torch.equal(c.backward(want_dx=False)[1], dw)
    y, z = c.forward()
    assert torch.equal(c.forward(keep=False)[0], y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_graph_replays_follow_the_offsets(dtype):
    c = Case([200, 0, 56, 100], 128, 128, True, dtype=dtype, seed=7)
    other = Case([1, 300, 50, 5], 128, 128, True, dtype=dtype, seed=8)
    c.forward(), c.backward()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = c.forward() + c.backward()
    graph.replay()
    c.check_forward(*out[:2])
    c.check_backward(*out[2:])
    c.bounds, c.sizes = other.bounds, other.sizes
    c.offsets.copy_(other.offsets)
    c.w.copy_(other.w)
    graph.replay()
    c.check_forward(*out[:2])
    c.check_backward(*out[2:])


@pytest.mark.gpu
def test_two_streams_with_their_own_workspaces():
    a = Case([130, 20, 300], 512, 256, True, seed=9)
    b = Case([7, 0, 2, 11], 512, 256, False, seed=10)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(5):
        outs = [(c.forward(stream=s), c.backward(stream=s)) for c, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for c, (f, g) in zip((a, b), outs):
        c.check_forward(*f)
        c.check_backward(*g)
    moe.sync_check()


@pytest.mark.gpu
@pytest.mark.parametrize("offsets", [[0, 50, 40, 90], [0, 50, 4000, 90], [-5, 30, 60, 90],
                                     [0, 2 ** 31 - 1, -2 ** 31, 90]])
def test_bad_offsets_are_held_and_reported(offsets):
    c = Case([30, 30, 30], 64, 64, False, seed=11)
    c.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    y, _ = c.forward()
    with pytest.raises(moe.MoEError):
        moe.sync_check()
    held, m = [], 0
    for o in offsets:
        m = max(m, min(max(o, 0), 90))
        held.append(m)
    for e in range(3):
        a, b = held[e], held[e + 1]
        ref = c.x[a:b].double() @ c.w[e * 64:(e + 1) * 64].double().t()
        assert_close(y[a:b], ref, HALF * ref.abs() + 1e-4)
    c.backward()
    with pytest.raises(moe.MoEError):
        moe.sync_check()
    moe.sync_check()


# ---------------------------------------------------------------------- refusals (CPU) ----

A = 0x7000_0000_0000  # never dereferenced: every call below fails validation first


def _cfg(**kw):
    base = dict(rows=64, groups=4, in_features=64, out_features=64)
    base.update(kw)
    return moe.GroupedConfig.make(**base)


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), INVALID), (dict(rows=2 ** 30 + 1), INVALID), (dict(groups=0), INVALID),
    (dict(groups=1025), INVALID), (dict(in_features=0), INVALID),
    (dict(out_features=0), INVALID), (dict(in_features=2 ** 18 + 1), INVALID),
    (dict(dtype=5), INVALID), (dict(out_dtype=moe.BF16, dtype=moe.F32), INVALID),
    (dict(dx_dtype=moe.BF16, dtype=moe.F32), INVALID), (dict(activation=9), INVALID),
    (dict(activation=-1), INVALID), (dict(activation=moe.ACT_GELU), UNSUPPORTED),
    (dict(x_stride=63), INVALID), (dict(z_stride=64, activation=moe.ACT_SWIGLU), INVALID),
    (dict(dw_stride=2 ** 31 + 1), INVALID),
    (dict(rows=2 ** 30, out_features=2 ** 18), UNSUPPORTED),
    (dict(groups=1024, in_features=2 ** 18, out_features=2 ** 18), UNSUPPORTED),
])
def test_bad_configs(bad, status):
    lib, n = moe.load(), ctypes.c_size_t(0)
    c = _cfg(**bad)
    assert lib.moe_grouped_linear_workspace_size(ctypes.byref(c), ctypes.byref(n)) == status


def test_bad_calls():
    lib, p = moe.load(), ctypes.c_void_p
    c = _cfg()
    need = moe.grouped_linear_workspace_size(c)
    assert need > 0

    def fwd(c=c, x=A, o=A, w=A, y=A, z=None, ws=A, n=None):
        return lib.moe_grouped_linear(ctypes.byref(c), p(x), p(o), p(w), p(y), p(z), p(ws),
                                      need if n is None else n, None)

    def bwd(c=c, dy=A, x=A, o=A, w=A, z=None, dx=A, dw=A, ws=A, n=None):
        return lib.moe_grouped_linear_backward(ctypes.byref(c), p(dy), p(x), p(o), p(w), p(z),
                                               p(dx), p(dw), p(ws), need if n is None else n, None)

    for kw in (dict(x=None), dict(o=None), dict(w=None), dict(y=None), dict(z=A)):
        assert fwd(**kw) == INVALID, kw
    for kw in (dict(x=A + 2), dict(w=A + 8), dict(o=A + 2), dict(y=A + 1), dict(ws=A + 8)):
        assert fwd(**kw) == MISALIGNED, kw
    assert fwd(ws=None) == WORKSPACE and fwd(n=need - 1) == WORKSPACE
    for kw in (dict(dy=None), dict(o=None), dict(x=None), dict(w=None), dict(dx=None, dw=None)):
        assert bwd(**kw) == INVALID, kw
    for kw in (dict(dy=A + 2), dict(x=A + 2), dict(w=A + 2), dict(dx=A + 1), dict(dw=A + 1)):
        assert bwd(**kw) == MISALIGNED, kw
    assert bwd(ws=None) == WORKSPACE and bwd(n=need - 1) == WORKSPACE
    s = _cfg(activation=moe.ACT_SWIGLU)
    assert bwd(c=s, n=1 << 40) == INVALID  # no z
    assert lib.moe_grouped_linear_workspace_size(ctypes.byref(c), None) == INVALID
    e = _cfg(rows=0)
    assert fwd(c=e, x=None, o=None, w=None, y=None, ws=None) == OK
    assert bwd(c=e, dy=None, x=None, o=None, w=None, dx=None, dw=None, ws=None) == OK


@pytest.mark.gpu
def test_no_rows_zero_the_weights_gradient():
    c = _cfg(rows=0)
    dw = torch.full((4 * 64, 64), 3.0, dtype=BF16, device="cuda")
    moe.grouped_linear_backward(c, None, None, None, None, None, None, dw)
    assert (dw == 0).all()
