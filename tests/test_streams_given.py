"""The ``stream`` argument of the operators around the attention.

CPU: a stream of another device than the tensors' is refused before any device work (the kernel
would run there, on this device's addresses).
"""

import types

import pytest

from block_sparse_attention_bigbird_b200 import bsa


def test_a_stream_of_another_device_is_refused(monkeypatch):
    import torch

    def never(*_):
        raise AssertionError("device work")
    monkeypatch.setattr(torch.cuda, "device", never)
    monkeypatch.setattr(torch.cuda, "stream", never)
    other = types.SimpleNamespace(device_index=1, cuda_stream=7)
    with pytest.raises(ValueError, match="another device"):
        bsa._on(0, other, never)
