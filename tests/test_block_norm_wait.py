"""A row that never arrives in block_norm's rings: the bounded wait for it ends the kernel with
MOE_ERR_TIMEOUT, whatever the row's threads and the block's other rows are doing then.

The fault is a barrier that lacks an arrival (moe_debug_set_fault), with a limit of 2 ms: nothing
faults and nothing waits for ever.  The threads of a row meet at a barrier in every row, so they have to
leave together; rows of one warp (which meet in a vote), of several warps, several rows a block and
rows that are not aligned are each taken once.
"""

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_block_norm import BF16, F32, Case

TIMEOUT = 5


@pytest.fixture(autouse=True)
def disarm():
    yield
    moe.debug_set_fault(None)


def times_out(point, call):
    moe.sync_check()
    moe.debug_set_fault(point, 1)
    call()
    moe.debug_set_fault(None)
    with pytest.raises(moe.MoEError) as e:
        moe.sync_check()
    assert e.value.status == TIMEOUT
    moe.sync_check()


@pytest.mark.parametrize("point", ["moe_block_norm.copy", "moe_block_norm_backward.copy"])
def test_the_points_are_known(point):
    moe.debug_set_fault(point, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width", [(9000, 64), (5000, 512), (4000, 1000), (2000, 2048),
                                        (700, 7168)])
def test_forward(rows, width, dtype):
    c = Case(rows, width, dtype, seed=width)
    want = c.forward()
    times_out("moe_block_norm.copy", c.forward)
    for a, b in zip(c.forward(), want):
        assert torch.equal(a, b)
    moe.sync_check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width", [(9000, 64), (5000, 512), (4000, 1000), (2000, 2048),
                                        (700, 4096), (9000, 65), (2000, 2047)])
def test_backward(rows, width, dtype):
    c = Case(rows, width, dtype, seed=width)
    want = c.backward()
    times_out("moe_block_norm_backward.copy", c.backward)
    for k, t in c.backward().items():
        assert torch.equal(t, want[k]), k
    moe.sync_check()
