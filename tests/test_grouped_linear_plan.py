"""The plan of grouped products: offsets that are not what they should be, in every kernel, and the
tiles of few rows that hold gate and up blocks in one box.

Offsets that descend or leave 0..rows are held to the largest before them and to rows: every result
is then that of the held bounds, and rows outside them stay as they were.  Tolerances are those of
test_grouped_linear.
"""

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_grouped_linear import BF16, F32, Case

pytestmark = pytest.mark.gpu

INTERNAL = 6


def hold(offsets, rows):
    held, most = [], 0
    for o in offsets:
        most = max(most, min(max(o, 0), rows))
        held.append(most)
    return held


BAD = [(0, 150, 100, 330, 390), (-7, 60, 9999, 200, 390), (20, 10, 5, 250, 2 ** 31 - 1),
       (0, 2 ** 31 - 1, -2 ** 31, 90, 395), (30, 140, 130, 135, 300), (400, 3, 2, 1, 0)]


@pytest.mark.parametrize("dtype,dx", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("fin,fout,pad", [(64, 128, 0), (65, 33, 1)])
# a mean of over 64 rows a group (CTA pairs, a table of tiles), of up to 64 and up to 32
@pytest.mark.parametrize("rows", [400, 200, 90])
@pytest.mark.parametrize("offsets", BAD, ids=str)
def test_bad_offsets_are_held(offsets, rows, fin, fout, pad, act, dtype, dx):
    offsets = [o if abs(o) > 1000 else o * rows // 400 for o in offsets]
    c = Case([rows // 4] * 4, fin, fout, act, dtype=dtype, dx=dx, pad=pad, seed=41)
    c.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    c.bounds = hold(offsets, rows)
    c.head = c.bounds[0]
    for e in range(4):
        if c.bounds[e] == c.bounds[e + 1]:
            c.w[e * c.N:(e + 1) * c.N] = float("nan")
    for call, check in ((c.forward, c.check_forward), (c.backward, c.check_backward)):
        out = call()
        with pytest.raises(moe.MoEError) as e:
            moe.sync_check()
        assert e.value.status == INTERNAL
        moe.sync_check()
        check(*out)


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("fin", [64, 200])
@pytest.mark.parametrize("fout", [16, 48, 80, 112, 144, 768, 1200, 5120])
@pytest.mark.parametrize("sizes", [[1], [1, 0, 1, 1, 1, 0, 1, 1], [3, 0, 20], [40, 60, 50]],
                         ids=str)
def test_gate_and_up_blocks_in_one_box(sizes, fout, fin, keep):
    """out_features that are multiples of 16, so that a tile's box ends inside the weights; 8 groups of
    768 and 1 of 5120 take tiles of 96 rows on 128 (or 107) to 159 SMs."""
    c = Case(sizes, fin, fout, True, tail=2, seed=fout)
    c.check_forward(*c.forward(keep=keep))
    moe.sync_check()


def test_the_sizes_above_take_every_tile():
    """The rule of the kernel, restated: 32 q rows of weights a tile, the least that goes round once."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    taken = set()
    for groups, rows, fout in ((1, 3, 16), (8, 8, 768), (1, 3, 5120), (8, 8, 1200)):
        active = min(groups, rows)
        q = next((q for q in (2, 3) if active * -(-fout // (16 * q)) <= sms), 4)
        taken.add(q)
    assert taken == {2, 3, 4}
