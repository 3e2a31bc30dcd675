"""BigBird block-sparse attention for B200 (sm_100a): forward and gradients, and the
operators around it (rotary positions, a block's norms and residual, 8-bit projections).

The compute lives in libbsa.so (C ABI, include/bsa.h); ``bsa`` is its thin
ctypes binding and ``autograd`` holds the torch.autograd forms.
Attributes are resolved lazily so that the build module can be imported before
the library exists; any other attribute access loads the library and fails
loudly if it is missing.
"""

from __future__ import annotations

import importlib

__all__ = ["bsa_layout_build", "bsa_layout_from_csr", "bsa_layout_csr", "bsa_layout_globals",
           "bsa_layout_tiles", "bsa_layout_key_tiles", "bsa_layout_upload", "bsa_workspace_bytes",
           "bsa_forward", "bsa_backward", "bsa_backward_workspace_bytes", "bsa_sync_status",
           "bsa_strerror", "bsa_debug_wait_timeout", "bsa_forward_static_ws", "Layout", "BsaError",
           "block_sparse_attention", "BigBirdSelfAttention",
           "bsa_rope_build", "bsa_rope_from_table", "bsa_rope_table", "bsa_rope_apply", "Rope",
           "bsa_block_norm", "bsa_block_norm_backward", "bsa_fp8_quantize", "bsa_fp8_matmul",
           "bsa_fp8_matmul_workspace_bytes", "rotary", "block_norm", "fp8_linear", "BigBirdBlock"]


def __getattr__(name):
    if name in ("block_sparse_attention", "rotary", "block_norm", "fp8_linear"):
        return getattr(importlib.import_module(".autograd", __name__), name)
    if name in ("BigBirdSelfAttention", "BigBirdBlock"):
        return getattr(importlib.import_module(".layer", __name__), name)
    if name in __all__:
        return getattr(importlib.import_module(".bsa", __name__), name)
    raise AttributeError(name)
