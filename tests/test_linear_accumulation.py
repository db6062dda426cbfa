"""How float32 results of linear layers are accumulated: partial sums leave the tensor core, whose
additions truncate, every 128 values of float32 operands and every 256 of bf16 ones, and are
then added with rounding.  Formulas as in tests/test_linear.py.
"""

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_linear import config, workspace


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,fin,fout", [(9, 14336, 64), (150, 14336, 64), (300, 4096, 200)])
def test_float32_sums_leave_the_tensor_core_every_128_values(rows, fin, fout):
    """Values of one sign, so that what the truncations lose adds up in the mean error of the
    results (whose own roundings, 2^-25 each, average out).  It is proportional to the run: with
    128 values (six products each) 3.8e-7 was measured, with 1024 1.9e-6 to 2.9e-6; for bf16
    operands 1.4e-8 with 256 and 7.3e-7 with 1024.  The limits lie between."""
    g = gen(fin)
    x = torch.rand(rows, fin, generator=g, device="cuda") + 0.5
    w = torch.rand(fout, fin, generator=g, device="cuda") + 0.5
    c = config(rows, fin, fout, dtype=moe.F32)
    y = torch.empty(rows, fout, device="cuda")
    moe.linear(c, x, w, None, None, y, None, workspace(c))
    want = x.double() @ w.double().t()
    rel = (y.double() - want) / want
    assert abs(rel.mean().item()) < 1e-6
    xb, wb = x.bfloat16(), w.bfloat16()
    c = config(rows, fin, fout, out_dtype=moe.F32)
    moe.linear(c, xb, wb, None, None, y, None, workspace(c))
    moe.sync_check()
    want = xb.double() @ wb.double().t()
    rel = (y.double() - want) / want
    assert abs(rel.mean().item()) < 1.5e-7
