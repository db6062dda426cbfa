"""What GradList takes and refuses, on the CPU: tensors that only say they are on a GPU."""

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe


class OnGpu:
    """As much of a GPU tensor as GradList asks for."""

    def __init__(self, at, n, dtype=torch.float32, device=0, contiguous=True):
        self.at, self.n, self.dtype, self.contiguous = at if n else 0, n, dtype, contiguous
        self.device, self.is_cuda = torch.device("cuda", device), True

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def element_size(self):
        return 2 if self.dtype == torch.bfloat16 else 4

    def is_contiguous(self):
        return self.contiguous


A = 0x7000_0000_0000


def test_empty_gradients_with_results_of_another_type():
    grads = [OnGpu(A, 8, torch.bfloat16), OnGpu(A, 0, torch.bfloat16)]
    outs = [OnGpu(A + 64, 8), OnGpu(A, 0)]
    lst = moe.GradList(grads, outs)
    assert len(lst) == 2 and [lst.array[i].size for i in (0, 1)] == [8, 0]
    assert (lst.array[1].dtype, lst.array[1].out_dtype) == (moe.BF16, moe.F32)
    with pytest.raises(ValueError):  # in place, with elements
        moe.GradList([OnGpu(A, 8, torch.bfloat16)], [OnGpu(A, 8)])


def test_tensors_of_two_gpus_are_refused():
    """One launch reads all of them: on another GPU that is a fault, or slow."""
    a, b = OnGpu(A, 8), OnGpu(A + 64, 8, device=1)
    for grads, outs in (([a, b], None), ([a], [b]), ([b], [a]), ([a, OnGpu(A + 128, 4)], [a, b])):
        with pytest.raises(ValueError):
            moe.GradList(grads, outs)
    moe.GradList([b, OnGpu(A + 128, 4, device=1)], None)
