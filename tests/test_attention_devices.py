"""Which tensors the attention's and the projections' bindings take, and on which device they run.

CPU: over meta tensors that say they are on a GPU, with the library's entry replaced: a tensor on
another device, or a result of another type, shape or layout, is refused before the library is
called (its kernels would read or write out of range); the tensors' own device is the current
one during the call.
"""

import contextlib
import types

import pytest
import torch

from block_sparse_attention_bigbird_b200 import bsa

B, H, L = 2, 3, 256


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)

    def get_device(self):
        return getattr(self, "index", 0)


def _t(*shape, dtype=torch.bfloat16, index=0):
    t = torch.empty(*shape, dtype=dtype, device="meta").as_subclass(OnGpu)
    t.index = index
    return t


@pytest.fixture
def calls(monkeypatch):
    """Names of the library's entries called, with the current device during each."""
    seen, now = [], dict(index=0)

    class Device(contextlib.AbstractContextManager):
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now["index"] = now["index"], self.index

        def __exit__(self, *_):
            now["index"] = self.before

    def entry(name):
        return lambda *_: seen.append((name, now["index"])) or 0
    names = ("bsa_forward", "bsa_forward_static_ws", "bsa_backward", "bsa_qkv_projection", "bsa_out_projection")
    monkeypatch.setattr(bsa, "lib", types.SimpleNamespace(
        **{n: entry(n) for n in names}, bsa_forward_workspace_bytes=lambda *_: 0, bsa_backward_workspace_bytes=lambda *_: 0))
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now["index"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: types.SimpleNamespace(cuda_stream=5))
    monkeypatch.setattr(bsa, "_raw_stream", lambda index: 5)
    return seen


def _entries(index=0):
    """name -> (entry, its tensors by name, those that may be left out)"""
    lay = types.SimpleNamespace(handle=None, _workspaces={})
    x = lambda *s, **k: _t(*s, index=index, **k)  # noqa: E731
    q, k, v, o, d = (x(B, H, L, 64) for _ in range(5))
    lse, mask, ws = x(B, H, L, dtype=torch.float32), x(B, L, dtype=torch.uint8), x(512, dtype=torch.uint8)
    heads = lambda *names: {n: x(B, H, L, 64) for n in names}  # noqa: E731
    more = dict(key_mask=mask, out=x(B, H, L, 64), lse=lse)
    return {
        "bsa_forward": (lambda **t: bsa.bsa_forward(layout=lay, **t), dict(q=q, k=k, v=v), {**more, "workspace": ws}),
        "bsa_forward_static_ws": (lambda **t: bsa.bsa_forward_static_ws(layout=lay, **t), dict(q=q, k=k, v=v), more),
        "bsa_backward": (lambda **t: bsa.bsa_backward(layout=lay, **t), dict(q=q, k=k, v=v, out=o, dout=d, lse=lse),
                         {"key_mask": mask, "workspace": ws, **heads("dq", "dk", "dv")}),
        "bsa_qkv_projection": (bsa.bsa_qkv_projection, dict(x=x(B, L, 64 * H), weight=x(192 * H, 64 * H)),
                               {"bias": x(192 * H), **heads("q", "k", "v")}),
        "bsa_out_projection": (bsa.bsa_out_projection, dict(o=o, weight=x(128, 64 * H)), dict(bias=x(128), y=x(B, L, 128))),
    }


NAMES = list(_entries())


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(calls, name):
    call, need, may = _entries()[name]
    call(**need)
    call(**need, **may)
    assert calls == [(name, 0)] * 2
    for which, t in {**need, **may}.items():
        for other in (_t(*t.shape, dtype=t.dtype, index=1), torch.empty(*t.shape, dtype=t.dtype)):
            with pytest.raises(ValueError):
                call(**{**need, **may, which: other})
    assert len(calls) == 2


@pytest.mark.parametrize("name", NAMES)
def test_results_that_do_not_fit_are_refused(calls, name):
    call, need, may = _entries()[name]
    for which, t in may.items():
        if which in ("workspace", "bias", "key_mask"):
            continue
        half = list(t.shape[:-1]) + [t.shape[-1] // 2]
        for other in (_t(*half, dtype=t.dtype), _t(*t.shape, dtype=torch.float16),
                      _t(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]):
            with pytest.raises(ValueError):
                call(**{**need, **may, which: other})
    assert not calls


@pytest.mark.parametrize("name", NAMES)
def test_the_tensors_device_is_the_current_one(calls, name):
    call, need, may = _entries(index=1)[name]
    call(**need, **may)
    assert calls == [(name, 1)]
    with pytest.raises(ValueError, match="another device"):
        call(**need, **may, stream=types.SimpleNamespace(device_index=0, cuda_stream=3))


def test_a_layers_layout_is_uploaded_to_its_inputs_device(calls, monkeypatch):
    from block_sparse_attention_bigbird_b200 import BigBirdSelfAttention
    monkeypatch.setattr(bsa, "bsa_layout_build", lambda *_: types.SimpleNamespace())
    monkeypatch.setattr(bsa, "bsa_layout_upload", lambda _: calls.append(("upload", torch.cuda.current_device())))
    layer = BigBirdSelfAttention(128, 2)
    for device in ("cuda:1", "cuda:0", "cuda:1"):
        layer.layout(64, torch.device(device))
    assert calls == [("upload", 1), ("upload", 0)]
