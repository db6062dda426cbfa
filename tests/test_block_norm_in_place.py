"""block_norm in place: where it is refused, and the rows that are read again in each pass."""

import ctypes

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_block_norm import BF16, F32, Case

INVALID = 1
A, B, C, D = (0x7000_0000_0000 + (k << 32) for k in range(4))  # never dereferenced


def test_another_stride_in_place_is_refused():
    lib, p = moe.load(), ctypes.c_void_p

    def fwd(x, res, sum_, **strides):
        c = moe.BlockNormConfig.make(4, 64, **strides)
        return lib.moe_block_norm(ctypes.byref(c), p(x), p(res), None, None, None, p(D), p(sum_),
                                  p(C), None)

    def bwd(dsum, dx, dres, **strides):
        c = moe.BlockNormConfig.make(4, 64, **strides)
        return lib.moe_block_norm_backward(ctypes.byref(c), None, p(dsum), None, None, None, None,
                                           None, None, p(dx), p(dres), None, None, None, None, None,
                                           0, None)

    assert fwd(A, B, A, x_stride=72) == INVALID
    assert fwd(A, B, A, sum_stride=72) == INVALID
    assert fwd(A, B, B, residual_stride=72, sum_stride=80) == INVALID
    assert bwd(A, A, B, dx_stride=72) == INVALID
    assert bwd(A, B, A, sum_stride=72) == INVALID
    assert bwd(A, B, A, sum_stride=72, dx_stride=72) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("width,pad", [(8200, 0), (9001, 3), (20000, 8)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_rows(dtype, width, pad):
    c = Case(30, width, dtype, pad=pad, seed=8)
    s0, y0 = c.forward()
    for over in ("x", "res"):
        ins = {k: torch.zeros(30, width + pad, dtype=dtype, device="cuda") for k in ("x", "res")}
        for k in ins:
            ins[k][:, :width] = getattr(c, k)
        y = c.matrix()
        moe.block_norm(c.cfg, ins["x"], ins["res"], c.post, c.gate, c.scale, c.norm, ins[over], y)
        assert torch.equal(ins[over][:, :width], s0[:, :width]) and torch.equal(y, y0)
    want = c.backward()
    for over in (0, 1):
        outs = [c.matrix(), c.matrix()]
        ds = torch.zeros(30, width + pad, dtype=dtype, device="cuda")
        ds[:, :width] = c.ds
        outs[over] = ds
        moe.block_norm_backward(c.cfg, c.dy, ds, c.x, c.s, c.post, c.gate, c.scale, c.norm, *outs,
                                None, None, None, None, None)
        assert torch.equal(outs[0][:, :width], want["dx"][:, :width])
        assert torch.equal(outs[1][:, :width], want["dres"][:, :width])
