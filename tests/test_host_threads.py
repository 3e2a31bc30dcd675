"""Calls from several host threads at once, each on a stream of its own.

GPU: threads whose calls run one kernel with unlike sizes of shared memory: every call succeeds
and its results equal, bit by bit, those of the same call made alone.
"""

import sys
import threading

import pytest
import torch

from block_sparse_attention_bigbird_b200 import bsa

gpu = pytest.mark.gpu
needs_cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")


def _at_once(calls, times):
    """Runs each call `times` times in a thread and stream of its own; its last results, lists."""
    torch.cuda.synchronize()
    start, got, raised = threading.Barrier(len(calls)), [None] * len(calls), []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                for _ in range(times):
                    got[i] = calls[i]()
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            raised.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)  # a call ends while another is under way as often as can be
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    assert not raised, raised[:1]
    return got


def _same(got, want):
    assert all(all(torch.equal(a, b) for a, b in zip(g, w)) for g, w in zip(got, want))


def _product(K):  # a few tokens
    g = torch.Generator(device="cuda").manual_seed(K)
    a, w = (torch.randn(n, K, generator=g, device="cuda") for n in (4, 256))
    a, b = bsa.bsa_fp8_quantize(a), bsa.bsa_fp8_quantize(w, square=True)
    return lambda: [bsa.bsa_fp8_matmul(*a, *b)]


@gpu
@needs_cuda
@pytest.mark.parametrize("Ks", [(1024, 2048), (1000, 2000)])  # a warp for each block of 128 of K, up to 16
def test_products_of_a_few_rows(Ks):
    calls = [_product(K) for K in Ks * 2]
    want = [c() for c in calls]
    _same(_at_once(calls, 8000), want)
    assert bsa.bsa_sync_status() == 0


def _norm(C, back):
    g = torch.Generator(device="cuda").manual_seed(C)
    x, y, ds, dn = torch.randn(4, 16, C, generator=g, device="cuda").unbind(0)
    a = dict(post="rms", pre="rms", post_weight=torch.rand(C, generator=g, device="cuda"),
             pre_weight=torch.rand(C, generator=g, device="cuda"))
    s, n, st = bsa.bsa_block_norm(x, y, save_stats=True, **a)
    if not back:
        return lambda: list(bsa.bsa_block_norm(x, y, save_stats=True, **a))
    return lambda: [v for v in bsa.bsa_block_norm_backward(ds, dn, s, y, st, **a).values() if v is not None]


@gpu
@needs_cuda
@pytest.mark.parametrize("back", [False, True])
def test_block_norms_of_unlike_widths(back):
    calls = [_norm(C, back) for C in (1024, 4096, 1024, 4096)]
    want = [c() for c in calls]
    _same(_at_once(calls, 6000), want)
