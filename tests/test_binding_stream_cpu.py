"""The binding's default stream is torch's current one, with or without the quick way to it."""

import types

import pytest
import torch

import mixture_experts_layer_04_gb300 as moe


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_a_torch_without_the_raw_handle_falls_back(monkeypatch, missing):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 11, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda *a: types.SimpleNamespace(cuda_stream=42))
    assert moe._stream(None) == 11
    monkeypatch.delattr(torch._C, missing)
    assert moe._stream(None) == 42


def test_given_streams_are_taken_as_they_are():
    assert moe._stream(7) == 7 and moe._stream(0) == 0
    assert moe._stream(types.SimpleNamespace(cuda_stream=9)) == 9


@pytest.mark.gpu
def test_the_default_follows_torchs_current_stream():
    assert moe._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert moe._stream(None) == side.cuda_stream
