"""Grouped products whose arrays start off a 16-byte boundary: results always may, operands where their
row stride is no multiple of 16 bytes (they are packed then).  What lies before and behind an array
stays as it was.  Tolerances are those of test_grouped_linear.
"""

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_grouped_linear import BF16, F32, Case

pytestmark = pytest.mark.gpu


class Shifted(Case):
    """Arrays `shift` elements into their storage, which holds 7 around them."""

    def __init__(self, *args, shift=1, **kw):
        self.shift, self.stores = shift, []
        super().__init__(*args, **kw)
        for name in ("x", "w", "dy", "z"):
            t = getattr(self, name)
            if name == "z" or t.stride(0) * t.element_size() % 16 != 0:
                setattr(self, name, self._moved(t))

    def _store(self, rows, ld, dtype):
        flat = torch.full((rows * ld + 2 * self.shift,), 7.0, dtype=dtype, device="cuda")
        self.stores.append(flat)
        return flat[self.shift:self.shift + rows * ld].view(rows, ld)

    def _moved(self, t):
        to = self._store(t.shape[0], t.stride(0), t.dtype)
        to[:, :t.shape[1]] = t
        return to[:, :t.shape[1]]

    def buffer(self, rows, cols, dtype):
        return self._store(rows, cols + self.pad, dtype)

    def check_around(self):
        for flat in self.stores:
            assert (flat[:self.shift] == 7).all() and (flat[-self.shift:] == 7).all()


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("fin,fout,pad", [(64, 128, 0), (200, 72, 8), (65, 33, 0), (130, 96, 1)])
@pytest.mark.parametrize("sizes", [[3, 0, 20], [40, 60], [300, 0, 70]], ids=str)
@pytest.mark.parametrize("shift", [1, 4])
def test_arrays_off_a_boundary(sizes, fin, fout, pad, act, dtype, out, shift):
    c = Shifted(sizes, fin, fout, act, dtype=dtype, out=out, dx=out, pad=pad, tail=2, head=1,
                seed=51, shift=shift)
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())
    c.check_around()
    moe.sync_check()
