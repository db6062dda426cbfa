"""moe_linear asks for a workspace only where it uses one: calls on the CUDA cores take NULL."""

import ctypes

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from mixture_experts_layer_04_gb300 import build as moe_build
from tests.test_linear import A, CUDA, UNSUPPORTED, WORKSPACE, config, make, workspace

FEW = [dict(rows=1, fin=4096, fout=4096), dict(rows=1, fin=7, fout=5, dtype=moe.F32),
       dict(rows=8, fin=4096, fout=4096, dtype=moe.F32), dict(rows=8, fin=100, fout=60),
       dict(rows=4, fin=512, fout=1024), dict(rows=6, fin=64, fout=64, x_stride=69)]
MORE = [dict(rows=9, fin=64, fout=64, dtype=moe.F32), dict(rows=5, fin=64, fout=64),
        dict(rows=4, fin=1024, fout=1024), dict(rows=9, fin=64, fout=64, x_stride=69)]


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def call(lib, c, ws=None, nb=0):
    return lib.moe_linear(ctypes.byref(c), A, A, None, None, A, None, ws, nb, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")
@pytest.mark.parametrize("kw", FEW)
def test_few_rows_are_not_refused_for_want_of_a_workspace(lib, kw):
    assert call(lib, config(**kw)) in (CUDA, UNSUPPORTED)


@pytest.mark.parametrize("kw", MORE)
def test_other_calls_still_are(lib, kw):
    c = config(**kw)
    assert call(lib, c) == WORKSPACE
    assert call(lib, c, A, moe.linear_workspace_size(c) - 1) == WORKSPACE


def test_the_size_is_never_zero(lib):
    for kw in FEW + MORE + [dict(rows=0)]:
        assert moe.linear_workspace_size(config(**kw)) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("kw", FEW)
def test_results_without_a_workspace_are_those_with_one(kw):
    c = config(activation=moe.ACT_SILU, **kw)
    dtype = torch.float32 if c.dtype == moe.F32 else torch.bfloat16
    pad = max(0, c.x_stride - c.in_features)
    x, w, b, res, _ = make(c.rows, c.in_features, c.out_features, dtype, 1, pad)
    out = [torch.full((c.rows, c.out_features), 7.0, dtype=dtype, device="cuda") for _ in range(4)]
    moe.linear(c, x, w, b, res, out[0], out[1], workspace(c))
    moe.linear(c, x, w, b, res, out[2], out[3])
    moe.sync_check()
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
