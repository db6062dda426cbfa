"""Grouped products, norms around a block and clipping where elements lie past 2^31 and 2^32 of their
array: the last rows (or groups) against 64 bits, and rows before them with the same inputs bit for
bit.  Tolerances: those of test_grouped_linear and test_block_norm, for the sizes checked.
"""

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_block_norm import Case as NormCase
from tests.test_grouped_linear import BF16, F32, HALF, acc, assert_close

pytestmark = pytest.mark.gpu

G32 = 1 << 32


def filled(g, rows, cols, dtype, block, std=1.0):
    """rows x cols whose rows repeat every `block`: quick to make, and its rows can be compared."""
    part = (torch.randn(block, cols, generator=g, device="cuda") * std).to(dtype)
    out = torch.empty(rows, cols, dtype=dtype, device="cuda")
    for at in range(0, rows, block):
        n = min(block, rows - at)
        out[at:at + n] = part[:n]
    return out


def test_grouped_rows():
    """Two groups of 300,000 and 300 rows of 16384 inputs."""
    g = torch.Generator(device="cuda").manual_seed(1)
    fin, fout, sizes = 16384, 64, (300000, 300)
    rows = sum(sizes)
    assert rows * fin > G32
    x = filled(g, rows, fin, BF16, 1000)
    w = (torch.randn(2 * fout, fin, generator=g, device="cuda") * fin ** -0.5).to(BF16)
    w[fout:] = w[:fout]
    offsets = torch.tensor([0, sizes[0], rows], dtype=torch.int32, device="cuda")
    cfg = moe.GroupedConfig.make(rows, 2, fin, fout, moe.BF16, moe.F32)
    ws = torch.empty(moe.grouped_linear_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    y = torch.empty(rows, fout, device="cuda")
    moe.grouped_linear(cfg, x, offsets, w, y, None, ws)
    a, b = x[-300:].double(), w[fout:].double().t()
    assert_close(y[-300:], a @ b, (a.abs() @ b.abs()) * (acc(fin, BF16) + 2.0 ** -24))
    assert torch.equal(y[:300], y[-300:])
    dy = filled(g, rows, fout, BF16, 1000)
    dx = torch.empty_like(x)
    dw = torch.empty_like(w)
    cfg = moe.GroupedConfig.make(rows, 2, fin, fout, moe.BF16)
    moe.grouped_linear_backward(cfg, dy, x, offsets, w, None, dx, dw, ws)
    a, b = dy[-300:].double(), w[fout:].double()
    assert_close(dx[-300:], a @ b, (a.abs() @ b.abs()) * acc(fout, BF16) + HALF * (a @ b).abs())
    assert torch.equal(dx[:300], dx[-300:])
    a, b = dy[-300:].double().t(), x[-300:].double()
    assert_close(dw[fout:], a @ b, (a.abs() @ b.abs()) * acc(300, BF16) + HALF * (a @ b).abs())
    moe.sync_check()


@pytest.mark.parametrize("sizes", [[0] * 126 + [5, 9], [0] * 126 + [100, 9900]], ids=["few", "many"])
def test_grouped_weights(sizes):
    """128 groups of 2 x 2560 x 8192 weights."""
    g = torch.Generator(device="cuda").manual_seed(2)
    fin, fout, groups = 8192, 2560, 128
    N, rows = 2 * fout, sum(sizes)
    assert groups * N * fin > G32
    w = filled(g, groups * N, fin, BF16, N, fin ** -0.5)
    x, dy = filled(g, rows, fin, BF16, rows), filled(g, rows, fout, BF16, rows)
    bounds = [0]
    for n in sizes:
        bounds.append(bounds[-1] + n)
    offsets = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    cfg = moe.GroupedConfig.make(rows, groups, fin, fout, moe.BF16, activation=moe.ACT_SWIGLU)
    ws = torch.empty(moe.grouped_linear_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    y, z = (torch.empty(rows, n, dtype=BF16, device="cuda") for n in (fout, N))
    moe.grouped_linear(cfg, x, offsets, w, y, z, ws)
    last = slice(bounds[-2], min(rows, bounds[-2] + 200))
    a, b = x[last].double(), w[-N:].double().t()
    assert_close(z[last], a @ b, (a.abs() @ b.abs()) * acc(fin, BF16) + HALF * (a @ b).abs())
    dx, dw = torch.empty_like(x), torch.full_like(w, 7.0)
    moe.grouped_linear_backward(cfg, dy, x, offsets, w, z, dx, dw, ws)
    assert (dw[:126 * N] == 0).all() if rows < 100 else (dw[:N] == 0).all()
    all_last = slice(bounds[-2], rows)
    gate, up = z[all_last, :fout].double(), z[all_last, fout:].double()
    s = torch.sigmoid(gate)
    d = dy[all_last].double()
    dz = torch.cat([d * up * (s + gate * s * (1 - s)), d * gate * s], dim=1)
    a, b = dz[:, -64:].t(), x[all_last].double()  # the last rows of the last group
    assert_close(dw[-64:], a @ b, (a.abs() @ b.abs()) * (acc(b.shape[0], BF16) + HALF + 4e-5) * 1.01
                 + HALF * (a @ b).abs() + 1e-37)
    a, b = dz[:200], w[-N:].double()
    assert_close(dx[last], a @ b, (a.abs() @ b.abs()) * (acc(N, BF16) + HALF + 4e-5) * 1.01
                 + HALF * (a @ b).abs() + 1e-37)
    moe.sync_check()


@pytest.mark.parametrize("width", [8192, 4095, 8200])
def test_norm_rows(width):
    """Rows in a ring, unaligned ones and those read again; the first ones are the last ones."""
    rows = G32 // width + 500
    block = 1000
    c = NormCase(block, width, BF16, seed=3)
    first = (rows - block) % block  # so that the last block of rows is the first, shifted
    names = ("x", "res", "s", "ds", "dy")

    def long(t):
        out = torch.empty(rows, *t.shape[1:], dtype=t.dtype, device="cuda")
        out[:first] = t[block - first:]
        for at in range(first, rows, block):
            out[at:at + block] = t
        return out

    d = NormCase(1, width, BF16, seed=3)
    for n in names + ("gate",):
        setattr(d, n, long(getattr(c, n)))
    d.post, d.scale, d.norm = c.post, c.scale, c.norm
    d.rows, d.cfg.rows = rows, rows
    want = c.forward()
    got = d.forward()
    for a, b in zip(got, want):
        assert torch.equal(a[-block:], b) and torch.equal(a[first:first + block], b)
    del got
    want = c.backward(outs="xrg", ws=False)
    got = d.backward(outs="xrg", ws=False)
    for k in ("dx", "dres", "dg"):
        assert torch.equal(got[k][-block:], want[k])
        assert torch.equal(got[k][first:first + block], want[k])
    moe.sync_check()


def test_clip_one_tensor_of_more_than_32_bits():
    n = G32 + 12345
    grad = torch.empty(n, dtype=BF16, device="cuda")
    grad.fill_(0.5)
    grad[-1] = 4.0
    out = torch.full((n,), 7.0, dtype=BF16, device="cuda")
    lst = moe.GradList([grad], [out])
    ws = torch.empty(moe.clip_grad_norm_workspace_size(lst), dtype=torch.uint8, device="cuda")
    norm = torch.zeros(1, device="cuda")
    moe.clip_grad_norm(lst, 1e9, norm, ws, grad_scale=0.25)
    want = 0.25 * ((n - 1) * 0.25 + 16.0) ** 0.5
    assert abs(norm.item() / want - 1) < 5 * 2.0 ** -24
    assert out[-1].item() == 1.0 and (out[:-1] == 0.125).all()
