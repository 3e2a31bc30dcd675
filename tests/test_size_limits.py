"""Sizes past the C interface's 32-bit integers, which ctypes would cut without a word.

CPU: shapes without storage behind them (meta tensors that say they are on a GPU); every binding
refuses them before it asks for memory or calls the library.
"""

import pytest
import torch

from block_sparse_attention_bigbird_b200 import bsa

BIG = 2 ** 32 + 3  # cut to 32 bits it would be 3
E4 = torch.float8_e4m3fn


class OnGpu(torch.Tensor):
    def get_device(self):
        return 0


def _t(*shape, dtype=torch.bfloat16, pitch=None):
    t = torch.empty(*shape, dtype=dtype, device="meta")
    if pitch is not None:
        t = torch.empty_strided(shape, (pitch, 1), dtype=dtype, device="meta")
    return t.as_subclass(OnGpu)


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def never(*_):
        raise AssertionError("the call went on")
    monkeypatch.setattr(bsa, "_on", never)


@pytest.mark.parametrize("B,H,Hk,L,d", [(1, 1, 1, BIG, 2), (BIG, 1, 0, 1, 2), (1, BIG, 0, 1, 2), (1, 1, BIG, 1, 2),
                                        (1, 1, 1, 1, BIG)])
def test_rotary(B, H, Hk, L, d):
    rope = bsa.bsa_rope_build([1])
    q, k = _t(B, H, L, d), _t(B, Hk, L, d) if Hk else None
    with pytest.raises(ValueError, match="31 bits"):
        bsa.bsa_rope_apply(q, k, _t(1, B, L, dtype=torch.int64), rope)


@pytest.mark.parametrize("shape", [(BIG, 1), (2, BIG, 1), (1, BIG)])
def test_block_norm(shape):
    x = _t(*shape)
    with pytest.raises(ValueError, match="31 bits"):
        bsa.bsa_block_norm(x)
    with pytest.raises(ValueError, match="31 bits"):
        bsa.bsa_block_norm_backward(None, x, x, None, _t(x.numel() // shape[-1], 4, dtype=torch.float32))


@pytest.mark.parametrize("shape", [(BIG, 1), (1, BIG), (2, BIG, 4)])
def test_quantiser(shape):
    with pytest.raises(ValueError, match="31 bits"):
        bsa.bsa_fp8_quantize(_t(*shape))


@pytest.mark.parametrize("M,N,K", [(BIG, 4, 16), (4, BIG, 16), (4, 4, BIG)])
def test_product(M, N, K):
    ld = (K + 15) // 16 * 16
    a, b = _t(M, K, dtype=E4, pitch=ld), _t(N, K, dtype=E4, pitch=ld)
    sa, sb = (_t(n, (K + 127) // 128, dtype=torch.float32) for n in (M, N))
    with pytest.raises(ValueError, match="31 bits"):
        bsa.bsa_fp8_matmul(a, sa, b, sb)
    with pytest.raises(ValueError, match="31 bits"):
        bsa.bsa_fp8_matmul_workspace_bytes(M, N, K)
