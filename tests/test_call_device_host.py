"""The library launches on the current device: a call whose tensors or stream are of another
one is refused before anything is launched (its kernels would run where the tensors are not)."""
from __future__ import annotations

import types

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa


@pytest.fixture
def two_devices(monkeypatch):
    now = [0]
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(msa, "_devices", 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    return now


def test_tensors_on_another_device(two_devices):
    one, two = torch.device("cuda", 0), torch.device("cuda", 1)
    assert msa._stream(one, None) == 100
    with pytest.raises(ValueError, match="current device"):
        msa._stream(two, None)
    two_devices[0] = 1
    assert msa._stream(two, None) == 101
    with pytest.raises(ValueError, match="current device"):
        msa._stream(one, None)


def test_stream_of_another_device(two_devices):
    one, two = torch.device("cuda", 0), torch.device("cuda", 1)
    stream = types.SimpleNamespace(cuda_stream=7, device_index=0)
    assert msa._stream(one, stream) == 7
    two_devices[0] = 1
    for dev in (one, two):
        with pytest.raises(ValueError):
            msa._stream(dev, stream)
    stream.device_index = 1
    assert msa._stream(two, stream) == 7
