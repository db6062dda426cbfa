"""The norms around a block, its gate and residual scale, against 64-bit torch, forward and backward.

Tolerances.  Every value of a row is a product of a few float32 factors and a sum of two terms, so it
is off by a few 2^-24 of the terms' sizes (8 are allowed: FEW); a root mean square over n values,
summed in float32 over lanes and warps, by (n / 256 + 12) 2^-24 of itself (a thread adds up to 64
values, 10 steps across lanes and warps), which is also what a row's dot product is off by, of the
sum of its products' sizes.  An output is rounded once more: 2^-8 of itself in bf16, 2^-24 in
float32.  Column sums of n rows: a thread adds up to n / 152 rows, then blocks: (n / 152 + 64) 2^-24
of the sum of sizes, each term off by FEW and its row's sums.
"""

import ctypes

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe

OK, INVALID, WORKSPACE, MISALIGNED = 0, 1, 3, 7
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {BF16: moe.BF16, F32: moe.F32}
GATES = {"none": moe.GATE_NONE, "value": moe.GATE_VALUE, "logistic": moe.GATE_LOGISTIC}
E = 2.0 ** -24
FEW = 8 * E
EPS = 1e-6


def row_sums(width):
    return (width / 256 + 12) * E


def step(dtype):
    return 2.0 ** -8 if dtype == BF16 else E


def assert_close(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), got.double()[bad][:4].tolist(),
                           ref[bad][:4].tolist(), tol.expand_as(ref)[bad][:4].tolist())


class Case:
    def __init__(self, rows, width, dtype=BF16, post=True, gate="logistic", scale=True,
                 residual=True, norm=True, pad=0, seed=0, ar=0.875, ab=0.75):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.width, self.dtype, self.pad = rows, width, dtype, pad
        self.gate_kind, self.ar, self.ab = gate, ar, ab

        def mat():
            size = torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
            return (torch.randn(rows, width + pad, generator=g, device="cuda") * size).to(dtype)[
                :, :width]

        def vec(on, n=width, mean=1.0):
            v = mean + 0.3 * torch.randn(n, generator=g, device="cuda")
            return v if on else None

        self.x, self.res = mat(), mat() if residual else None
        self.post, self.scale, self.norm = vec(post), vec(scale), vec(norm)
        self.gate = None if gate == "none" else vec(True, rows, 0.0 if gate == "logistic" else 1.0)
        self.s, self.ds, self.dy = mat(), mat(), mat() if norm else None
        ld = width + pad
        self.cfg = moe.BlockNormConfig.make(
            rows, width, TYPES[dtype], EPS, ar, ab, GATES[gate], ld, ld, ld, ld, ld, ld)

    def matrix(self, on=True):
        return torch.full((self.rows, self.width + self.pad), 7.0, dtype=self.dtype,
                          device="cuda") if on else None

    def forward(self, want_sum=True, **kw):
        sum_, y = self.matrix(want_sum), self.matrix(self.norm is not None)
        moe.block_norm(self.cfg, self.x, self.res, self.post, self.gate, self.scale, self.norm,
                       sum_, y, **kw)
        return sum_, y

    def _terms(self):
        d = lambda t: None if t is None else t.double()
        x, g = d(self.x), d(self.gate)
        one = torch.ones((), dtype=torch.float64, device="cuda")
        rx = 1 / (x.pow(2).mean(1, keepdim=True) + EPS).sqrt() if self.post is not None else one
        g = one if g is None else (g.sigmoid() if self.gate_kind == "logistic" else g)[:, None]
        sc = one if self.scale is None else d(self.scale)
        wp = one if self.post is None else d(self.post)
        return x, rx, g, sc, wp

    def check_forward(self, sum_, y):
        W = self.width
        x, rx, g, sc, wp = self._terms()
        a = self.ab * g * sc * x * rx * wp
        b = self.ar * self.res.double() if self.res is not None else torch.zeros_like(a)
        s = a + b
        off = (FEW + row_sums(W)) * (a.abs() + b.abs())
        for t in (sum_, y):
            if t is not None:
                assert (t[:, W:] == 7).all()
        if sum_ is not None:
            assert_close(sum_[:, :W], s, off + step(self.dtype) * s.abs(), "sum")
        if y is not None:
            r = 1 / (s.pow(2).mean(1, keepdim=True) + EPS).sqrt()
            w = self.norm.double()
            # R moves by no more than the relative error of the mean square: 2 |s| off / W, summed
            shift = (s.abs() * off).mean(1, keepdim=True) * r * r
            ref = s * r * w
            tol = (off * r * w.abs() + ref.abs() * (shift + FEW + row_sums(W) + step(self.dtype)))
            assert_close(y[:, :W], ref, tol, "y")

    def backward(self, dy=True, dsum=True, outs="xrgpsn", ws=True, **kw):
        f = lambda on, n: torch.full((n,), 7.0, device="cuda") if on else None
        dx, dres = self.matrix("x" in outs), self.matrix("r" in outs)
        has = lambda k, v: k in outs and v is not None
        dg = f(has("g", self.gate), self.rows)
        dp, dsc = f(has("p", self.post), self.width), f("s" in outs, self.width)
        dn = f(has("n", self.norm) and dy, self.width)
        buf = torch.full((moe.block_norm_workspace_size(self.cfg),), 255, dtype=torch.uint8,
                         device="cuda") if ws else None
        moe.block_norm_backward(self.cfg, self.dy if dy else None, self.ds if dsum else None,
                                self.x, self.s, self.post, self.gate, self.scale, self.norm, dx,
                                dres, dg, dp, dsc, dn, buf, **kw)
        return dict(dx=dx, dres=dres, dg=dg, dp=dp, dsc=dsc, dn=dn)

    def check_backward(self, got, dy=True, dsum=True):
        W, n = self.width, self.rows
        x, rx, g, sc, wp = self._terms()
        rel = FEW + row_sums(W)
        ds = self.ds.double() if dsum else torch.zeros_like(x)
        size = ds.abs()
        if dy and self.dy is not None:
            s, d, w = self.s.double(), self.dy.double(), self.norm.double()
            r = 1 / (s.pow(2).mean(1, keepdim=True) + EPS).sqrt()
            u = s * r
            cols = d * u
            ds = ds + r * (d * w - u * (d * w * u).mean(1, keepdim=True))
            size = size + r * ((d * w).abs() + u.abs() * (d * w * u).abs().mean(1, keepdim=True))
        off = 2 * rel * size
        out = step(self.dtype)
        c = self.ab * sc * wp
        summed = (n / 152 + 64) * E
        mats = dict(dx=None, dres=(self.ar * ds, abs(self.ar) * (off + out * ds.abs())))
        p, q = x * rx, ds * c
        dq = off * c.abs()
        dot, dot_size = (q * p).sum(1), (q * p).abs().sum(1)
        dot_off = (dq * p.abs()).sum(1) + 2 * rel * dot_size
        if self.post is not None:
            v = g * rx * (q - p * dot[:, None] / W)
            v_off = (g * rx).abs() * (dq + p.abs() * dot_off[:, None] / W
                                      + 2 * rel * (q.abs() + p.abs() * dot_size[:, None] / W))
        else:
            v, v_off = g * q, g.abs() * (dq + 2 * rel * q.abs())
        mats["dx"] = (v, v_off + out * v.abs())
        for name, (ref, tol) in mats.items():
            if got[name] is not None:
                assert (got[name][:, W:] == 7).all()
                assert_close(got[name][:, :W], ref, tol, name)
        if got["dg"] is not None:
            slope = torch.ones(n, dtype=torch.float64, device="cuda")
            if self.gate_kind == "logistic":
                slope = g[:, 0] * (1 - g[:, 0])
            assert_close(got["dg"], dot * slope, (dot_off + FEW * dot_size) * slope, "dgate")
        a = g * ds * p
        a_off = (g * p).abs() * off + 2 * rel * a.abs()
        for name, f in (("dp", self.ab * sc), ("dsc", self.ab * wp)):
            if got[name] is not None:
                f = f * torch.ones(W, dtype=torch.float64, device="cuda")
                assert_close(got[name], a.sum(0) * f,
                             (a_off + (summed + FEW) * a.abs()).sum(0) * f.abs(), name)
        if got["dn"] is not None:
            assert_close(got["dn"], cols.sum(0), ((summed + 2 * rel) * cols.abs()).sum(0), "dnorm")


SHAPES = [(1, 7168), (3, 64), (700, 8), (5, 1), (33, 2048), (1000, 512), (2, 8192), (3, 8200),
          (2, 40000), (7, 65536), (400, 257), (9, 5287), (1500, 96)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_all_parts(rows, width, dtype):
    c = Case(rows, width, dtype, seed=rows)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width,pad", [(64, 8), (65, 0), (1001, 5), (2048, 4), (9000, 3)])
def test_strides(width, pad, dtype):
    c = Case(50, width, dtype, pad=pad, seed=width)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


@pytest.mark.gpu
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "value", "logistic"])
@pytest.mark.parametrize("scale", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_parts_left_out(post, gate, scale, residual, norm):
    for width in (768, 20000):
        c = Case(21, width, BF16, post, gate, scale, residual, norm, seed=3)
        c.check_forward(*c.forward())
        c.check_backward(c.backward())
        if norm:
            c.check_forward(*c.forward(want_sum=False))
            c.check_backward(c.backward(dsum=False), dsum=False)
        c.check_backward(c.backward(dy=False), dy=False)
        everything = c.backward()
        for one, there in (("x", True), ("r", True), ("g", gate != "none"), ("p", post),
                           ("s", True), ("n", norm)):
            if there:  # each output by itself is what it is among the others
                for name, t in c.backward(outs=one, ws=one in "psn").items():
                    if t is not None:
                        assert torch.equal(t, everything[name]), (one, name)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [48, 64, 96, 184, 192, 368, 376, 384, 512, 1536])
def test_many_rows_of_every_number_of_arrays(width):
    """Rings of 46 to 48 KB among them, which need more shared memory than a launch has by default."""
    for dtype in (BF16, F32):
        for residual in (False, True):
            c = Case(5000, width, dtype, residual=residual, seed=width)
            c.check_forward(*c.forward())
            c.check_backward(c.backward())
            c.check_backward(c.backward(dsum=False), dsum=False)
            c.check_backward(c.backward(dy=False), dy=False)
            c.post = c.gate = None  # x is not read: one array, or two
            c.cfg.gate, c.gate_kind = moe.GATE_NONE, "none"
            c.check_backward(c.backward(outs="xr", ws=False))
            c.check_backward(c.backward(outs="xr", ws=False, dy=False), dy=False)


def embedded(t, width, start, pad):
    """t's rows of `width` in a buffer of NaN, `start` values into it and `pad` apart."""
    flat = torch.full((start + t.shape[0] * (width + pad) + 8,), float("nan"), dtype=t.dtype,
                      device="cuda")
    rows = flat[start:start + t.shape[0] * (width + pad)].view(t.shape[0], width + pad)
    rows[:, :width] = t[:, :width]
    return rows[:, :width]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width,pad", [(15, 0), (16, 1), (17, 0), (33, 2), (64, 3), (255, 0),
                                       (257, 0), (511, 4), (512, 1), (513, 0), (1001, 5),
                                       (2047, 0), (2048, 1), (4095, 0), (4097, 0), (5287, 0),
                                       (8191, 0)])
def test_many_unaligned_rows(width, pad, dtype):
    """Their copies take pieces of the neighbouring rows along, which hold NaN here."""
    rows = 5000 if width < 1000 else 700
    for start in (0, 3):
        for residual in (False, True):
            c = Case(rows, width, dtype, residual=residual, pad=pad, seed=width)
            for name in ("x", "res", "s", "ds", "dy"):
                t = getattr(c, name)
                if t is not None:
                    setattr(c, name, embedded(t, width, start, pad))
            c.check_forward(*c.forward())
            c.check_backward(c.backward())
            c.check_backward(c.backward(dsum=False), dsum=False)
            c.check_backward(c.backward(dy=False), dy=False)
            c.check_backward(c.backward(outs="xr", ws=False))


@pytest.mark.gpu
@pytest.mark.parametrize("width", [1001, 2047])
def test_many_unaligned_rows_in_place(width):
    c = Case(2000, width, BF16, seed=8)
    s0, y0 = c.forward()
    for over in ("x", "res"):
        ins = dict(x=c.x.clone(), res=c.res.clone())
        y = c.matrix()
        moe.block_norm(c.cfg, ins["x"], ins["res"], c.post, c.gate, c.scale, c.norm, ins[over], y)
        assert torch.equal(ins[over], s0) and torch.equal(y, y0)
    want = c.backward()
    for over in (0, 1):
        outs = [c.matrix(), c.matrix()]
        outs[over] = ds = c.ds.clone()
        moe.block_norm_backward(c.cfg, c.dy, ds, c.x, c.s, c.post, c.gate, c.scale, c.norm, *outs,
                                None, None, None, None, None)
        assert torch.equal(outs[0], want["dx"]) and torch.equal(outs[1], want["dres"])


@pytest.mark.gpu
def test_gradients_against_differences():
    c = Case(3, 40, F32, seed=5, ab=1.25)
    g = torch.Generator(device="cuda").manual_seed(6)
    ds, dy = (torch.randn(3, 40, generator=g, device="cuda", dtype=torch.float64) for _ in range(2))

    def value(x, res, gate, post, scale, norm):
        p = x / (x.pow(2).mean(1, keepdim=True) + EPS).sqrt() * post
        s = c.ar * res + c.ab * gate.sigmoid()[:, None] * scale * p
        y = s / (s.pow(2).mean(1, keepdim=True) + EPS).sqrt() * norm
        return (s * ds).sum() + (y * dy).sum()

    ins = [t.double() for t in (c.x, c.res, c.gate, c.post, c.scale, c.norm)]
    p = ins[0] / (ins[0].pow(2).mean(1, keepdim=True) + EPS).sqrt() * ins[3]
    c.s = (c.ar * ins[1] + c.ab * ins[2].sigmoid()[:, None] * ins[4] * p).float()
    c.ds, c.dy = ds.float(), dy.float()
    got = c.backward()
    h = 1e-5
    for k, name in enumerate(("dx", "dres", "dg", "dp", "dsc", "dn")):
        flat = ins[k].reshape(-1)
        num = torch.empty_like(flat)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = value(*ins)
            flat[i] = keep - h
            num[i] = (up - value(*ins)) / (2 * h)
            flat[i] = keep
        # differences of a float64 value near 100: 1e-14 / 1e-5, and h^2 times third derivatives;
        # the operator's inputs are float32 roundings (2^-24) of a sum of up to 40 terms near 5
        assert_close(got[name].reshape(-1), num, torch.full_like(num, 2e-4), name)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [256, 20000])
def test_in_place(width):
    c = Case(30, width, BF16, seed=8)
    s0, y0 = c.forward()
    stream_, y = c.res.clone(), c.matrix()
    moe.block_norm(c.cfg, c.x, stream_, c.post, c.gate, c.scale, c.norm, stream_, y)
    assert torch.equal(stream_, s0) and torch.equal(y, y0)
    x = c.x.clone()
    moe.block_norm(c.cfg, x, c.res, c.post, c.gate, c.scale, c.norm, x, y)
    assert torch.equal(x, s0) and torch.equal(y, y0)
    want = c.backward()
    dx, dres = c.matrix(), c.ds.clone()
    moe.block_norm_backward(c.cfg, c.dy, dres, c.x, c.s, c.post, c.gate, c.scale, c.norm, dx, dres,
                            None, None, None, None, None)
    assert torch.equal(dres, want["dres"]) and torch.equal(dx, want["dx"])


@pytest.mark.gpu
def test_rows_of_zeros_and_of_one_infinity():
    c = Case(4, 512, F32, seed=9)
    c.x[1] = 0
    c.res[1] = 0
    c.x[2, 7] = float("inf")
    sum_, y = c.forward()
    assert (sum_[1] == 0).all() and (y[1] == 0).all()
    keep = torch.tensor([0, 1, 3], device="cuda")
    d = Case(4, 512, F32, seed=9)
    d.x[1] = 0
    d.res[1] = 0
    for a, b in zip((sum_, y), d.forward()):
        assert torch.equal(a[keep], b[keep])
    big = Case(2, 64, F32, gate="logistic", seed=10)
    big.gate.copy_(torch.tensor([200.0, -200.0]))
    s, _ = big.forward()
    assert torch.isfinite(s).all()
    dg = big.backward()["dg"]
    assert torch.isfinite(dg).all()


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    c = Case(300, 1024, BF16, seed=11)
    want = c.forward(), c.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.forward(), c.backward()
    for t in list(out[0]) + list(out[1].values()):
        t.zero_()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = c.forward(), c.backward()
    torch.cuda.synchronize()
    for o in (out, again):
        for a, b in zip(o[0], want[0]):
            assert torch.equal(a, b)
        for k in want[1]:
            assert torch.equal(o[1][k], want[1][k]), k


# ---------------------------------------------------------------------- refusals (CPU) ----

A = 0x7000_0000_0000  # never dereferenced: every call below fails validation first


def _cfg(**kw):
    base = dict(rows=4, width=64)
    base.update(kw)
    return moe.BlockNormConfig.make(**base)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=2 ** 30 + 1), dict(width=0), dict(width=65537), dict(dtype=3),
    dict(gate=3), dict(gate=-1), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(residual_scale=float("nan")), dict(branch_scale=float("inf")), dict(x_stride=63),
    dict(dresidual_stride=2 ** 31 + 1),
])
def test_bad_configs(bad):
    n = ctypes.c_size_t(0)
    c = _cfg(**bad)
    assert moe.load().moe_block_norm_workspace_size(ctypes.byref(c), ctypes.byref(n)) == INVALID


def test_bad_calls():
    lib, p = moe.load(), ctypes.c_void_p
    plain, gated = _cfg(), _cfg(gate=moe.GATE_VALUE)
    need = moe.block_norm_workspace_size(plain)

    def fwd(c=plain, x=A, res=A, post=A, gate=None, scale=A, norm=A, sum_=A, y=A):
        return lib.moe_block_norm(ctypes.byref(c), *map(p, (x, res, post, gate, scale, norm, sum_,
                                                            y)), None)

    names = ("dy", "dsum", "x", "sum_", "post", "gate", "scale", "norm", "dx", "dres", "dg", "dp",
             "dsc", "dn")

    def bwd(c=plain, ws=A, n=need, **kw):
        args = {k: None if k in ("gate", "dg") else A for k in names}
        args.update(kw)
        return lib.moe_block_norm_backward(ctypes.byref(c), *[p(args[k]) for k in names], p(ws), n,
                                           None)

    for kw in (dict(x=None), dict(sum_=None, y=None, norm=None), dict(gate=A), dict(c=gated),
               dict(norm=None), dict(y=None)):
        assert fwd(**kw) == INVALID, kw
    for kw in (dict(x=A + 1), dict(res=A + 1), dict(post=A + 2), dict(scale=A + 1),
               dict(norm=A + 2), dict(sum_=A + 1), dict(y=A + 1)):
        assert fwd(**kw) == MISALIGNED, kw
    assert fwd(c=_cfg(rows=0), x=None, sum_=None, y=None) == OK
    for kw in (dict(dy=None, dsum=None), dict(sum_=None), dict(norm=None), dict(gate=A),
               dict(c=gated), dict(dg=A), dict(post=None), dict(dy=None), dict(x=None),
               dict(dx=None, dres=None, dp=None, dsc=None, dn=None)):
        assert bwd(**kw) == INVALID, kw
    for kw in (dict(dy=A + 1), dict(dx=A + 1), dict(dn=A + 2), dict(ws=A + 8)):
        assert bwd(**kw) == MISALIGNED, kw
    assert bwd(ws=None) == WORKSPACE and bwd(n=need - 1) == WORKSPACE
    none = {k: None for k in names}
    assert bwd(c=_cfg(rows=0), ws=None, **none) == OK


@pytest.mark.gpu
def test_no_rows_zero_the_vectors():
    c = _cfg(rows=0)
    v = [torch.full((64,), 3.0, device="cuda") for _ in range(3)]
    moe.block_norm_backward(c, *[None] * 11, *v)
    assert all((t == 0).all() for t in v)
