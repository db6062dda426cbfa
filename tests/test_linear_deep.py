"""Linear layers with bf16 results over very deep reductions (dW of a million rows, say).

The tensor core truncates its additions, and always the same way for values of one sign: a sum
that stays in one accumulator was measured to be low by 6.2e-9 of its size per value, 3e-3 over
524288.  An accumulator takes 16384 values at most, 1.0e-4, and partial sums are added with
rounding.  The columns' sizes are spread over a factor of two, so that the one rounding of each
result (under 2^-8, 1.7e-3 in the root mean square) averages to 2.6e-5 over 4096 of them.
"""

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_linear import config

MEAN = 3e-4            # 1.0e-4, and seven times 2.6e-5
EACH = 2.0 ** -8 + 4e-4
CUT = 64


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def positive(g, rows, cols, down=False):
    """Values of 0.5 to 1.5 times a factor of 1 to 2 per column (or row)."""
    f = 2.0 ** torch.rand(*((rows, 1) if down else (cols,)), generator=g, device="cuda")
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 1 << 18):
        n = min(1 << 18, rows - r)
        part = torch.rand(n, cols, generator=g, device="cuda") + 0.5
        out[r:r + n] = part * (f[r:r + n] if down else f)
    return out


def compare(got, want):
    rel = (got.double() - want) / want
    assert abs(rel.mean().item()) < MEAN
    assert (rel.abs() <= EACH).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,fin,fout", [((1 << 22) + 77, 64, 200), (1 << 21, 72, 64),
                                           ((1 << 19) + 5, 2048, 2048), (1 << 17, 2056, 2100),
                                           (1 << 15, 2048, 2048), (16384 + 64, 2048, 2048)])
def test_weight_gradients_over_many_rows(rows, fin, fout):
    g = gen(rows)
    x, dy = positive(g, rows, fin), positive(g, rows, fout)
    c = config(rows, fin, fout)
    dw = torch.empty(fout, fin, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(moe.linear_workspace_size(c), dtype=torch.uint8, device="cuda")
    moe.linear_backward(c, dy, x, None, None, None, dw, None, ws)
    moe.sync_check()
    for a, b in ((slice(0, CUT), slice(0, CUT)), (slice(fout - CUT, fout), slice(fin - CUT, fin))):
        want = torch.zeros(CUT, CUT, device="cuda", dtype=torch.float64)
        for r in range(0, rows, 1 << 19):
            s = slice(r, r + (1 << 19))
            want += dy[s, a].double().t() @ x[s, b].double()
        compare(dw[a, b], want)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,fin,fout", [(24, 1 << 20, 64), (100, (1 << 20) - 8, 72),
                                           (2048, 1 << 17, 2048), (2100, 16384 + 72, 2056)])
def test_forward_over_many_features(rows, fin, fout):
    g = gen(fout)
    x, w = positive(g, rows, fin, True), positive(g, fout, fin, True)
    c = config(rows, fin, fout, activation=moe.ACT_RELU)
    b = torch.rand(fout, generator=g, device="cuda")
    res = positive(g, rows, fout)
    y, z = torch.empty_like(res), torch.empty_like(res)
    ws = torch.empty(moe.linear_workspace_size(c), dtype=torch.uint8, device="cuda")
    moe.linear(c, x, w, b, res, y, z, ws)
    moe.sync_check()
    for i, j in ((slice(0, CUT), slice(0, CUT)), (slice(-CUT, rows), slice(-CUT, fout))):
        want = x[i].double() @ w[j].double().t() + b[j].double()
        compare(z[i, j], want)
        compare(y[i, j], want + res[i, j].double())


@pytest.mark.gpu
def test_deep_sums_of_both_signs_and_their_bits():
    # the error of ordinary data stays that of the one rounding, and calls repeat bit for bit
    rows, fin, fout = (1 << 17) + 3, 2048, 2048
    g = gen(9)
    x = torch.randn(rows, fin, generator=g, device="cuda").bfloat16()
    dy = torch.randn(rows, fout, generator=g, device="cuda").bfloat16()
    c = config(rows, fin, fout)
    ws = torch.empty(moe.linear_workspace_size(c), dtype=torch.uint8, device="cuda")
    dw, again = (torch.empty(fout, fin, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    moe.linear_backward(c, dy, x, None, None, None, dw, None, ws)
    moe.linear_backward(c, dy, x, None, None, None, again, None, ws)
    moe.sync_check()
    assert torch.equal(dw, again)
    want = dy[:, :256].double().t() @ x.double()
    assert (dw[:256].double() - want).norm() <= 2.0 ** -8 / 3 ** 0.5 * 1.05 * want.norm()
