"""The ``stream`` argument of the operators around the attention.

CPU: a stream of another device than the tensors' is refused before any device work (the kernel
would run there, on this device's addresses).
GPU: the default stream, given as its pointer 0, is the stream that the calls wait in.
"""

import types

import pytest
import torch

from block_sparse_attention_bigbird_b200 import bsa

gpu = pytest.mark.gpu
needs_cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")


def test_a_stream_of_another_device_is_refused(monkeypatch):
    def never(*_):
        raise AssertionError("device work")
    monkeypatch.setattr(torch.cuda, "device", never)
    monkeypatch.setattr(torch.cuda, "stream", never)
    other = types.SimpleNamespace(device_index=1, cuda_stream=7)
    with pytest.raises(ValueError, match="another device"):
        bsa._on(0, other, never)


@gpu
@needs_cuda
def test_the_default_stream_by_its_pointer():
    assert bsa._on(0, 0, lambda ptr: ptr) == 0
    rope = bsa.bsa_rope_build([32])
    pos = torch.arange(64, device="cuda")[None]
    ones = torch.ones(4, 4, 64, 64, device="cuda")
    calls = [lambda x: bsa.bsa_rope_apply(x, x, pos, rope, stream=0)[0], lambda x: bsa.bsa_block_norm(x, x, stream=0)[0],
             lambda x: bsa.bsa_fp8_quantize(x, stream=0)[1],
             lambda x: bsa.bsa_fp8_matmul(*(bsa.bsa_fp8_quantize(x, stream=0) * 2), stream=0)]
    want = [c(ones) for c in calls]
    torch.cuda.synchronize()
    for call, w in zip(calls, want):
        x = torch.zeros_like(ones)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # about 10 ms: a call that does not wait reads zeros
        x.fill_(1)
        got = call(x)
        torch.cuda.synchronize()
        assert torch.equal(got, w)


@gpu
@needs_cuda
def test_streams_of_every_kind():
    s, taken = torch.cuda.Stream(), lambda given: bsa._on(0, given, lambda ptr: (ptr, torch.cuda.current_stream().cuda_stream))  # noqa: E731
    foreign = types.SimpleNamespace(cuda_stream=s.cuda_stream)  # another library's stream object
    for given in (s, s.cuda_stream, foreign, torch.cuda.ExternalStream(s.cuda_stream)):
        assert taken(given) == (s.cuda_stream, s.cuda_stream)
    with torch.cuda.stream(s):
        assert taken(None) == taken(s) == taken(s.cuda_stream) == (s.cuda_stream, s.cuda_stream)
        assert taken(0) == taken(torch.cuda.default_stream()) == (0, 0)
    assert taken(None) == taken(0) == (0, 0) and torch.cuda.current_stream().cuda_stream == 0
