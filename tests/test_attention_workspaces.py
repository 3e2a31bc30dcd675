"""The workspaces that the binding keeps for bsa_forward and bsa_backward.

CPU: calls of one layout on one stream share a workspace; another stream has another, and a
captured call one of its own, which is not kept.
GPU: one layout on two streams at once, and two captured graphs of it replayed at once, forward and
backward, equal to the calls made alone.
"""

import types

import pytest
import torch

from block_sparse_attention_bigbird_b200 import bsa

gpu = pytest.mark.gpu
needs_cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")


def test_a_workspace_belongs_to_a_stream_or_a_graph(monkeypatch):
    layout, now = types.SimpleNamespace(_workspaces={}), dict(stream=7, capturing=False)
    monkeypatch.setattr(bsa, "_stream_ptr", lambda s: now["stream"] if s is None else s)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    take = lambda size=256, **kw: bsa._workspace(layout, ("fwd", 2, 64), lambda: size, "cpu", kw.get("stream"))  # noqa: E731
    first = take()
    assert take() is first and first.numel() == 256
    other = take(stream=9)
    assert other is not first and take(stream=9) is other
    now["stream"] = 9
    assert take() is other
    now["capturing"] = True
    a, b = take(), take()
    assert len({id(t) for t in (first, other, a, b)}) == 4
    now["capturing"] = False
    assert take() is other
    assert bsa._workspace(layout, ("bwd", 2, 64), lambda: 128, "cpu", None).numel() == 128


def _case(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(2, 2, 64 * 64, 64, generator=g, device="cuda").bfloat16() for _ in range(4)]


def _run(lay, q, k, v, d):
    out, lse = bsa.bsa_forward(q, k, v, lay)
    return [out, lse, *bsa.bsa_backward(q, k, v, out, d, lse, lay)]


@gpu
@needs_cuda
def test_one_layout_on_two_streams_and_in_two_graphs():
    lay = bsa.bsa_layout_build(2, 64 * 64, 64, 1, 2, 2, 0)  # global rows are split: partial results in the workspace
    bsa.bsa_layout_upload(lay)
    cases = [_case(1), _case(2)]
    want = [_run(lay, *c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _run(lay, *cases[i])
    torch.cuda.synchronize()
    assert bsa.bsa_sync_status() == 0
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    graphs, held = [], []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(_run(lay, *c))
        graphs.append(graph)
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert bsa.bsa_sync_status() == 0
    assert all(torch.equal(a, b) for g, w in zip(held, want) for a, b in zip(g, w))
