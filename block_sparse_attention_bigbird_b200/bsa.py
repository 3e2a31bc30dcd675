"""Thin ctypes binding of libbsa.so (the C ABI in include/bsa.h).

Argument marshalling only: every step of the forward runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  If the
shared library is missing this module raises at import; there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import numpy as np

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbsa.so")

BSA_OK = 0
BSA_ERR_INVALID_ARG = -1
BSA_ERR_UNSUPPORTED = -2
BSA_ERR_CUDA = -3
BSA_ERR_LAYOUT_MISMATCH = -4
BSA_ERR_DEVICE_TIMEOUT = -5
BSA_ERR_OOM = -6
BSA_ERR_WORKSPACE = -7
BSA_ERR_STATIC_WORKSPACE = -8
STATIC_WORKSPACE_BYTES = 32 * 1024 * 1024  # BSA_STATIC_WORKSPACE_BYTES in include/bsa.h
SPLIT_THRESHOLD = 48  # BSA_SPLIT_THRESHOLD in include/bsa.h: longer tile unions are split

# bsa_type in include/bsa.h
BF16, FP16, FP32, E4M3, E5M2, INT32, INT64 = range(7)
NORMS = {None: 0, "rms": 1, "layer": 2}  # BSA_NORM_*
NORM_COLUMNS_MOST = 8192
INT_MOST = 2 ** 31 - 1  # ctypes cuts what is above to 32 bits without a word


class BlockNormArgs(ctypes.Structure):
    """bsa_block_norm_args in include/bsa.h."""
    _fields_ = [("B", ctypes.c_int), ("rows_per_batch", ctypes.c_int), ("C", ctypes.c_int), ("type", ctypes.c_int),
                ("param_type", ctypes.c_int), ("post", ctypes.c_int), ("pre", ctypes.c_int),
                ("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("pre_weight", ctypes.c_void_p), ("pre_bias", ctypes.c_void_p), ("gate_rows", ctypes.c_int),
                ("branch_scale", ctypes.c_float), ("stream_scale", ctypes.c_float), ("eps", ctypes.c_float)]


# name -> (restype, argtypes); mirrors include/bsa.h
_SIGNATURES = {
    "bsa_layout_build": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, ctypes.c_uint64,
                                        ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_void_p)]),
    "bsa_layout_build_tokens": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                               ctypes.c_int, ctypes.c_uint64, ctypes.POINTER(ctypes.c_int32),
                                               ctypes.POINTER(ctypes.c_void_p)]),
    "bsa_layout_token_masks": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int),
                                              ctypes.POINTER(ctypes.c_void_p)]),
    "bsa_layout_from_csr": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                           ctypes.POINTER(ctypes.c_void_p)]),
    "bsa_layout_csr": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p),
                                      ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_int64),
                                      ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "bsa_layout_globals": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p),
                                          ctypes.POINTER(ctypes.c_int)]),
    "bsa_layout_tiles": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p),
                                        ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_void_p),
                                        ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_int64)]),
    "bsa_layout_upload": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "bsa_layout_free": (None, [ctypes.c_void_p]),
    "bsa_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int,
                                           ctypes.POINTER(ctypes.c_size_t)]),
    "bsa_forward_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                                   ctypes.POINTER(ctypes.c_size_t)]),
    "bsa_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                   ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "bsa_forward_static_ws": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p]),
    "bsa_layout_key_tiles": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p),
                                            ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_void_p),
                                            ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_int64)]),
    "bsa_backward_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int,
                                                    ctypes.POINTER(ctypes.c_size_t)]),
    "bsa_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                    ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]),
    "bsa_qkv_projection": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                          ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p]),
    "bsa_out_projection": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                          ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                          ctypes.c_void_p]),
    "bsa_rope_build": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32), ctypes.c_int, ctypes.c_double, ctypes.c_int,
                                      ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)]),
    "bsa_rope_from_table": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_double),
                                           ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)]),
    "bsa_rope_table": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p),
                                      ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_int),
                                      ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "bsa_rope_free": (None, [ctypes.c_void_p]),
    "bsa_rope_apply": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "bsa_block_norm": (ctypes.c_int, [ctypes.POINTER(BlockNormArgs), ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "bsa_block_norm_backward_workspace_bytes": (ctypes.c_int, [ctypes.POINTER(BlockNormArgs),
                                                               ctypes.POINTER(ctypes.c_size_t)]),
    "bsa_block_norm_backward": (ctypes.c_int, [ctypes.POINTER(BlockNormArgs)] + [ctypes.c_void_p] * 13 +
                                [ctypes.c_size_t, ctypes.c_void_p]),
    "bsa_fp8_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "bsa_fp8_matmul_workspace_bytes": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                      ctypes.POINTER(ctypes.c_size_t)]),
    "bsa_fp8_matmul": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int,
                                      ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int,
                                      ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_void_p]),
    "bsa_sync_status": (ctypes.c_int, [ctypes.c_void_p]),
    "bsa_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "bsa_debug_wait_timeout": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_void_p]),
    "bsa_debug_product_wait_timeout": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_void_p]),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing; build it with "
                          "`python -m block_sparse_attention_bigbird_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()
LIB_PATH = _LIB_PATH


class BsaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {bsa_strerror(code)} ({code})")
        self.code = code


def bsa_strerror(code: int) -> str:
    return lib.bsa_strerror(int(code)).decode()


def _check(code: int, what: str) -> None:
    if code != BSA_OK:
        raise BsaError(code, what)


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Layout:
    """Owner of a bsa_layout*; freed with the object."""

    def __init__(self, handle: int, H: int, L: int):
        self._h = ctypes.c_void_p(handle)
        self.H = H
        self.L = L
        self._workspaces = {}

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and lib is not None:   # lib is None at interpreter exit
            lib.bsa_layout_free(h)
            self._h = ctypes.c_void_p(0)


def bsa_layout_build(H: int, L: int, block: int = 64, window: int = 1, n_global: int = 2,
                     n_random: int = 3, seed: int = 0, globals=None) -> Layout:
    out = ctypes.c_void_p()
    gptr = None
    if globals is not None:
        g = np.ascontiguousarray(np.asarray(globals, dtype=np.int32))
        n_global = int(g.size)
        gptr = g.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    _check(lib.bsa_layout_build(H, L, block, window, n_global, n_random,
                                ctypes.c_uint64(seed & 0xFFFFFFFFFFFFFFFF), gptr, ctypes.byref(out)),
           "bsa_layout_build")
    return Layout(out.value, H, L)


def bsa_layout_build_tokens(H: int, L: int, window: int, n_global: int = 0, n_random: int = 0, seed: int = 0,
                            global_tokens=None) -> Layout:
    """A BigBird layout with its window and global set in tokens (see bsa.h)."""
    out = ctypes.c_void_p()
    gptr = None
    if global_tokens is not None:
        g = np.ascontiguousarray(np.asarray(global_tokens, dtype=np.int32))
        n_global = int(g.size)
        gptr = g.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    _check(lib.bsa_layout_build_tokens(H, L, window, n_global, n_random,
                                       ctypes.c_uint64(seed & 0xFFFFFFFFFFFFFFFF), gptr, ctypes.byref(out)),
           "bsa_layout_build_tokens")
    return Layout(out.value, H, L)


def bsa_layout_token_masks(layout: Layout):
    """(window in tokens, uint64 [L / 64] global-token bits) of a token-level layout."""
    w, gb = ctypes.c_int(), ctypes.c_void_p()
    _check(lib.bsa_layout_token_masks(layout.handle, ctypes.byref(w), ctypes.byref(gb)), "bsa_layout_token_masks")
    bits = np.ctypeslib.as_array(ctypes.cast(gb, ctypes.POINTER(ctypes.c_uint64)), (layout.L // 64,)).copy()
    return w.value, bits


def bsa_layout_from_csr(H: int, L: int, row_ptr, col_idx, block: int = 64) -> Layout:
    """Layout from a caller's block CSR (rows head-major; see bsa_layout_from_csr in bsa.h)."""
    rp = np.ascontiguousarray(np.asarray(row_ptr, dtype=np.int32))
    ci = np.ascontiguousarray(np.asarray(col_idx, dtype=np.int32))
    if rp.ndim != 1 or rp.size != H * (L // block if block > 0 else 0) + 1:
        raise BsaError(BSA_ERR_INVALID_ARG, "bsa_layout_from_csr: row_ptr must hold H * L / block + 1 entries")
    if int(rp[-1]) > ci.size:
        raise BsaError(BSA_ERR_INVALID_ARG, "bsa_layout_from_csr: col_idx is shorter than row_ptr[-1]")
    out = ctypes.c_void_p()
    cptr = ci.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)) if ci.size else None
    _check(lib.bsa_layout_from_csr(H, L, block, rp.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), cptr,
                                   ctypes.byref(out)), "bsa_layout_from_csr")
    return Layout(out.value, H, L)


def bsa_layout_csr(layout: Layout):
    """(row_ptr int32 [H*nb+1], col_idx int32 [nnz]) as numpy copies."""
    rp, ci = ctypes.c_void_p(), ctypes.c_void_p()
    nnz, nb, H = ctypes.c_int64(), ctypes.c_int(), ctypes.c_int()
    _check(lib.bsa_layout_csr(layout.handle, ctypes.byref(rp), ctypes.byref(ci), ctypes.byref(nnz),
                              ctypes.byref(nb), ctypes.byref(H)), "bsa_layout_csr")
    n_rows = H.value * nb.value + 1
    row_ptr = np.ctypeslib.as_array(ctypes.cast(rp, ctypes.POINTER(ctypes.c_int32)), (n_rows,)).copy()
    col_idx = (np.ctypeslib.as_array(ctypes.cast(ci, ctypes.POINTER(ctypes.c_int32)), (nnz.value,)).copy()
               if nnz.value else np.zeros(0, np.int32))
    return row_ptr, col_idx


def bsa_layout_globals(layout: Layout) -> np.ndarray:
    gp, n = ctypes.c_void_p(), ctypes.c_int()
    _check(lib.bsa_layout_globals(layout.handle, ctypes.byref(gp), ctypes.byref(n)), "bsa_layout_globals")
    if n.value == 0:
        return np.zeros(0, np.int32)
    return np.ctypeslib.as_array(ctypes.cast(gp, ctypes.POINTER(ctypes.c_int32)), (n.value,)).copy()


def bsa_layout_tiles(layout: Layout):
    """(pair_q [n_pairs, 2], pair_ptr [H*n_pairs+1], pair_ent [n_ent] uint32) as numpy copies."""
    pq, pp, pe = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    n_pairs, n_ent = ctypes.c_int(), ctypes.c_int64()
    _check(lib.bsa_layout_tiles(layout.handle, ctypes.byref(pq), ctypes.byref(n_pairs), ctypes.byref(pp),
                                ctypes.byref(pe), ctypes.byref(n_ent)), "bsa_layout_tiles")
    P = n_pairs.value
    pair_q = np.ctypeslib.as_array(ctypes.cast(pq, ctypes.POINTER(ctypes.c_int32)), (2 * P,)).copy()
    pair_ptr = np.ctypeslib.as_array(ctypes.cast(pp, ctypes.POINTER(ctypes.c_int32)),
                                     (layout.H * P + 1,)).copy()
    pair_ent = np.ctypeslib.as_array(ctypes.cast(pe, ctypes.POINTER(ctypes.c_uint32)), (n_ent.value,)).copy()
    return pair_q.reshape(P, 2), pair_ptr, pair_ent


def bsa_layout_key_tiles(layout: Layout):
    """(pair_k [n_pairs, 2], pair_ptr [H*n_pairs+1], pair_ent [n_ent] uint32) of the key-major tiles."""
    pq, pp, pe = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    n_pairs, n_ent = ctypes.c_int(), ctypes.c_int64()
    _check(lib.bsa_layout_key_tiles(layout.handle, ctypes.byref(pq), ctypes.byref(n_pairs), ctypes.byref(pp),
                                    ctypes.byref(pe), ctypes.byref(n_ent)), "bsa_layout_key_tiles")
    P = n_pairs.value
    pair_k = np.ctypeslib.as_array(ctypes.cast(pq, ctypes.POINTER(ctypes.c_int32)), (2 * P,)).copy()
    pair_ptr = np.ctypeslib.as_array(ctypes.cast(pp, ctypes.POINTER(ctypes.c_int32)),
                                     (layout.H * P + 1,)).copy()
    pair_ent = np.ctypeslib.as_array(ctypes.cast(pe, ctypes.POINTER(ctypes.c_uint32)), (n_ent.value,)).copy()
    return pair_k.reshape(P, 2), pair_ptr, pair_ent


def bsa_layout_upload(layout: Layout, stream=None) -> None:
    _check(lib.bsa_layout_upload(layout.handle, ctypes.c_void_p(_stream_ptr(stream))), "bsa_layout_upload")
    layout._workspaces.clear()


def bsa_workspace_bytes(layout: Layout, B: int) -> int:
    n = ctypes.c_size_t()
    _check(lib.bsa_workspace_bytes(layout.handle, B, ctypes.byref(n)), "bsa_workspace_bytes")
    return n.value


def bsa_forward_workspace_bytes(layout: Layout, B: int, d: int) -> int:
    n = ctypes.c_size_t()
    _check(lib.bsa_forward_workspace_bytes(layout.handle, B, d, ctypes.byref(n)), "bsa_forward_workspace_bytes")
    return n.value


def _workspace(layout: Layout, key, size, device, stream):
    """A workspace of size() bytes for calls of one kind (``key``) on ``stream``: kept for later calls
    on that stream, which run one after the other; a captured call gets its own, which its
    graph holds, as graphs may run at once."""
    import torch
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(size(), dtype=torch.uint8, device=device)
    key = (*key, str(device), _stream_ptr(stream))
    ws = layout._workspaces.get(key)
    if ws is None:
        layout._workspaces[key] = ws = torch.empty(size(), dtype=torch.uint8, device=device)
    return ws


def _fits(name, t, shape, dtype, dev):
    """Refuses a tensor that is not a contiguous [shape] of this type on device dev."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor {list(shape)} on the inputs' device")


def _attention_inputs(q, k, v, key_mask, out, lse, workspace):
    """Refuses what bsa_forward does not take; (B, H, L, d, device index)."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor [B, H, L, d]")
    shape, dev = q.shape, q.get_device()
    if shape != k.shape or shape != v.shape:
        raise ValueError("q, k, v shapes differ")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k, v are on different devices")
    _attention_more(shape, dev, key_mask, workspace)
    if out is not None:
        _fits("out", out, shape, torch.bfloat16, dev)
    if lse is not None:
        _fits("lse", lse, shape[:3], torch.float32, dev)
    return *shape, dev


def _attention_more(shape, dev, key_mask, workspace):
    import torch
    if key_mask is not None:
        _fits("key_mask", key_mask, (shape[0], shape[2]), torch.uint8, dev)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous and on the inputs' device")


def _attention_outputs(q, out, lse):
    import torch
    return (torch.empty_like(q) if out is None else out,
            q.new_empty(q.shape[:3], dtype=torch.float32) if lse is None else lse)


def bsa_forward(q, k, v, layout: Layout, key_mask=None, scale: Optional[float] = None, out=None,
                lse=None, workspace=None, stream=None):
    """O (bf16 [B,H,L,d]) and lse (fp32 [B,H,L]) of the block-sparse attention.

    q, k, v: contiguous bf16 CUDA tensors [B, H, L, d], d = 64 or 128.  key_mask: optional
    uint8 CUDA tensor [B, L] (1 = keep).  workspace: optional uint8 CUDA tensor
    of at least bsa_workspace_bytes(layout, B) bytes, any contents; when
    omitted one that the layout keeps for the stream is used (a captured call
    has its own, held by its graph).
    """
    B, H, L, d, dev = _attention_inputs(q, k, v, key_mask, out, lse, workspace)

    def call(ptr):
        o, ls = _attention_outputs(q, out, lse)
        ws = workspace
        if ws is None:
            ws = _workspace(layout, ("fwd", B, d), lambda: bsa_forward_workspace_bytes(layout, B, d), q.device, ptr)
        code = lib.bsa_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, L, d, layout.handle, _ptr(key_mask),
                               scale if scale is not None else 0.0, o.data_ptr(), ls.data_ptr(), ws.data_ptr(),
                               ws.numel(), ptr)
        _check(code, "bsa_forward")
        return o, ls
    return _on(dev, stream, call)


def bsa_forward_static_ws(q, k, v, layout: Layout, key_mask=None, scale: Optional[float] = None,
                          out=None, lse=None, stream=None):
    """bsa_forward for callers that cannot allocate device memory.

    The library's built-in scratch buffer (STATIC_WORKSPACE_BYTES per device)
    replaces the workspace; nothing is allocated by the call itself (``out`` and
    ``lse`` must then be given by such a caller).  Calls on one device share that
    buffer: serialise them.  Raises BsaError(BSA_ERR_STATIC_WORKSPACE) when the
    problem needs more scratch than the buffer holds.
    """
    B, H, L, d, dev = _attention_inputs(q, k, v, key_mask, out, lse, None)

    def call(ptr):
        o, ls = _attention_outputs(q, out, lse)
        code = lib.bsa_forward_static_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, L, d, layout.handle,
                                         _ptr(key_mask), scale if scale is not None else 0.0, o.data_ptr(),
                                         ls.data_ptr(), ptr)
        _check(code, "bsa_forward_static_ws")
        return o, ls
    return _on(dev, stream, call)


def bsa_backward_workspace_bytes(layout: Layout, B: int) -> int:
    n = ctypes.c_size_t()
    _check(lib.bsa_backward_workspace_bytes(layout.handle, B, ctypes.byref(n)), "bsa_backward_workspace_bytes")
    return n.value


def bsa_backward(q, k, v, out, dout, lse, layout: Layout, key_mask=None, scale: Optional[float] = None,
                 dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dq, dk, dv (bf16 [B,H,L,64]) of the block-sparse attention for dL/dO = ``dout``.

    q, k, v, out, dout: contiguous bf16 CUDA tensors [B, H, L, 64]; out and lse
    (fp32 [B, H, L]) are the forward's results for the same inputs, layout,
    key_mask and scale.  workspace: optional uint8 CUDA tensor of at least
    bsa_backward_workspace_bytes(layout, B) bytes (no clearing needed); when
    omitted one that the layout keeps for the stream is used (a captured call
    has its own, held by its graph).
    """
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor [B, H, L, d]")
        if t.shape != q.shape:
            raise ValueError(f"{name} shape differs from q")
    shape, dev = q.shape, q.get_device()
    B, H, L, d = shape
    if any(t.get_device() != dev for t in (k, v, out, dout)):
        raise ValueError("q, k, v, out, dout are on different devices")
    _fits("lse", lse, shape[:3], torch.float32, dev)
    _attention_more(shape, dev, key_mask, workspace)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        if t is not None:
            _fits(name, t, shape, torch.bfloat16, dev)

    def call(ptr):
        grads = [torch.empty_like(q) if t is None else t for t in (dq, dk, dv)]
        ws = workspace
        if ws is None:
            ws = _workspace(layout, ("bwd", B), lambda: bsa_backward_workspace_bytes(layout, B), q.device, ptr)
        code = lib.bsa_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), dout.data_ptr(),
                                lse.data_ptr(), B, H, L, d, layout.handle, _ptr(key_mask),
                                scale if scale is not None else 0.0, *(t.data_ptr() for t in grads), ws.data_ptr(),
                                ws.numel(), ptr)
        _check(code, "bsa_backward")
        return tuple(grads)
    return _on(dev, stream, call)


def _check_bf16(name, t, dim):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != dim:
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor of {dim} dimensions")


def bsa_qkv_projection(x, weight, bias=None, num_heads: Optional[int] = None, q=None, k=None, v=None,
                       stream=None):
    """q, k, v = the heads of x W^T + bias, each bf16 [B, H, L, 64].

    x: bf16 [B, L, C] with C = 64 H; weight: bf16 [3C, C] (rows: the q features,
    then k, then v; within each, head h's 64 features at 64 h); bias: bf16 [3C]
    or None.  The library's tcgen05 GEMM writes the three outputs in the head
    layout directly.
    """
    import torch
    _check_bf16("x", x, 3)
    _check_bf16("weight", weight, 2)
    B, L, C = x.shape
    H = num_heads if num_heads is not None else C // 64
    if C != 64 * H or tuple(weight.shape) != (3 * C, C):
        raise ValueError("x must be [B, L, 64 H] and weight [3 C, C]")
    dev = x.get_device()
    _fits("weight", weight, (3 * C, C), torch.bfloat16, dev)
    if bias is not None:
        _fits("bias", bias, (3 * C,), torch.bfloat16, dev)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is not None:
            _fits(name, t, (B, H, L, 64), torch.bfloat16, dev)

    def call(ptr):
        outs = tuple(x.new_empty((B, H, L, 64)) if t is None else t for t in (q, k, v))
        code = lib.bsa_qkv_projection(x.data_ptr(), weight.data_ptr(), _ptr(bias), B, L, H,
                                      *(t.data_ptr() for t in outs), ptr)
        _check(code, "bsa_qkv_projection")
        return outs
    return _on(dev, stream, call)


def bsa_out_projection(o, weight, bias=None, y=None, stream=None):
    """y = merge_heads(o) W^T + bias, bf16 [B, L, N].

    o: bf16 [B, H, L, 64] (the attention output); weight: bf16 [N, 64 H] with N
    a multiple of 64; bias: bf16 [N] or None.  The heads are merged by the
    GEMM's own tile loads.
    """
    import torch
    _check_bf16("o", o, 4)
    _check_bf16("weight", weight, 2)
    B, H, L, d = o.shape
    N = weight.shape[0]
    if d != 64 or weight.shape[1] != 64 * H:
        raise ValueError("o must be [B, H, L, 64] and weight [N, 64 H]")
    dev = o.get_device()
    _fits("weight", weight, (N, 64 * H), torch.bfloat16, dev)
    if bias is not None:
        _fits("bias", bias, (N,), torch.bfloat16, dev)
    if y is not None:
        _fits("y", y, (B, L, N), torch.bfloat16, dev)

    def call(ptr):
        out = o.new_empty((B, L, N)) if y is None else y
        code = lib.bsa_out_projection(o.data_ptr(), weight.data_ptr(), _ptr(bias), B, H, L, N, out.data_ptr(), ptr)
        _check(code, "bsa_out_projection")
        return out
    return _on(dev, stream, call)


_type_codes = {}


def _type_of(dtype) -> Optional[int]:
    """bsa_type of a torch dtype, None for one the library has no name for."""
    if not _type_codes:
        import torch
        _type_codes.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32,
                            torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2, torch.int32: INT32,
                            torch.int64: INT64})
    return _type_codes.get(dtype)


_current_raw = None


def _raw_stream(index: int) -> int:
    """The current stream's pointer (without building a stream object, where torch allows)."""
    global _current_raw
    if _current_raw is None:
        import torch
        _current_raw = getattr(torch._C, "_cuda_getCurrentRawStream",
                               lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _current_raw(index)


def _on(index: int, stream, call):
    """call(stream pointer) with the tensors' device ``index`` current, and ``stream``, where one
    is given, the stream that call's allocations belong to.  An integer, or the ``cuda_stream`` of an
    object that is no torch stream, is taken to be a stream of that device."""
    import torch
    if stream is not None:
        if getattr(stream, "device_index", index) != index:
            raise ValueError("stream belongs to another device than the tensors")
        if not isinstance(stream, (int, torch.cuda.Stream)):
            stream = stream.cuda_stream
    if index == torch.cuda.current_device():
        ptr = _raw_stream(index)
        if stream is None or (stream if isinstance(stream, int) else stream.cuda_stream) == ptr:
            return call(ptr)
    with torch.cuda.device(index):
        if stream is None:
            return call(_raw_stream(index))
        if isinstance(stream, int):
            # torch makes a new stream of the pointer 0
            stream = torch.cuda.ExternalStream(stream, device=index) if stream else torch.cuda.default_stream(index)
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


_TOO_LARGE = "a size needs more than 31 bits"


# ---------------------------------------------------------------- rotary positions
class Rope:
    """Owner of a bsa_rope*; freed with the object."""

    def __init__(self, handle: int):
        self._h = ctypes.c_void_p(handle)
        n, a, adj = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        lib.bsa_rope_table(self._h, None, None, ctypes.byref(n), ctypes.byref(a), ctypes.byref(adj))
        self.n_pairs, self.n_axes, self.adjacent = n.value, a.value, bool(adj.value)

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def __reduce__(self):  # copied and stored by its tables, with the module that holds it
        axis, freq = bsa_rope_table(self)
        return bsa_rope_from_table, (axis, freq, self.adjacent)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and lib is not None:   # lib is None at interpreter exit
            lib.bsa_rope_free(h)
            self._h = ctypes.c_void_p(0)


def bsa_rope_build(sections, base: float = 10000.0, per_axis: bool = False, interleave: bool = False,
                   adjacent: bool = False) -> Rope:
    """A rotary code whose axis a (time, height, ..) turns sections[a] pairs of a head.

    Frequencies are base^(-j / n) over all n pairs, or with ``per_axis``
    base^(-i / sections[a]) for the i-th pair of each axis; ``interleave`` deals the
    pairs to the axes in turn; pair j holds columns j and n + j, or 2 j and 2 j + 1 with
    ``adjacent``.
    """
    s = np.ascontiguousarray(np.asarray(sections, dtype=np.int32).reshape(-1))
    out = ctypes.c_void_p()
    _check(lib.bsa_rope_build(s.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), s.size, base, int(per_axis),
                              int(interleave), int(adjacent), ctypes.byref(out)), "bsa_rope_build")
    return Rope(out.value)


def bsa_rope_from_table(axis, freq, adjacent: bool = False) -> Rope:
    """A rotary code from the axis and the frequency (radians per position) of each pair."""
    a = np.ascontiguousarray(np.asarray(axis, dtype=np.int32).reshape(-1))
    f = np.ascontiguousarray(np.asarray(freq, dtype=np.float64).reshape(-1))
    if a.size != f.size:
        raise BsaError(BSA_ERR_INVALID_ARG, "bsa_rope_from_table: axis and freq differ in length")
    out = ctypes.c_void_p()
    _check(lib.bsa_rope_from_table(a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                   f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), a.size, int(adjacent),
                                   ctypes.byref(out)), "bsa_rope_from_table")
    return Rope(out.value)


def bsa_rope_table(rope: Rope):
    """(axis int32 [n_pairs], freq float64 [n_pairs]) as numpy copies."""
    a, f = ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib.bsa_rope_table(rope.handle, ctypes.byref(a), ctypes.byref(f), None, None, None), "bsa_rope_table")
    n = (rope.n_pairs,)
    return (np.ctypeslib.as_array(ctypes.cast(a, ctypes.POINTER(ctypes.c_int32)), n).copy(),
            np.ctypeslib.as_array(ctypes.cast(f, ctypes.POINTER(ctypes.c_double)), n).copy())


_pack3, _pack12 = struct.Struct("3q").pack, struct.Struct("12q").pack  # host int64 arrays


def bsa_rope_apply(q, k, positions, rope: Rope, inverse: bool = False, q_out=None, k_out=None, stream=None):
    """q [B, H, L, d] and k [B, Hk, L, d] (or None) with their pairs turned by their positions.

    bf16, fp16 or fp32 CUDA tensors of any strides with contiguous columns (views of a packed
    projection too).  positions: int32, int64 or fp32 [axes, L], shared by the batch, or
    [axes, B, L].  ``inverse`` turns back (the gradient).  Results are new contiguous tensors,
    or q_out and k_out, which may be q and k themselves; other overlaps are not allowed (and
    refused where two of them start at one address).
    """
    dev, dtype = q.get_device(), q.dtype
    ty, pt = _type_of(dtype), _type_of(positions.dtype)
    if q.dim() != 4 or ty is None or ty > FP32 or dev < 0:
        raise ValueError("q must be a bf16, fp16 or fp32 CUDA tensor [B, H, L, d]")
    B, H, L, d = q.shape
    sb, sh, sl, sc = q.stride()
    if sc != 1 and d != 1:
        raise ValueError("q must have contiguous columns")
    Hk, ks = 0, None
    if k is not None:
        ks = k.stride()
        if k.dim() != 4 or k.dtype is not dtype or k.get_device() != dev or k.shape[0] != B or k.shape[2] != L or \
                k.shape[3] != d or (ks[3] != 1 and d != 1):
            raise ValueError("k must be like q, [B, Hk, L, d] with contiguous columns")
        Hk = k.shape[1]
    ps, n = positions.stride(), positions.shape
    if (B | H | Hk | L | d) > INT_MOST:
        raise ValueError(_TOO_LARGE)
    if pt not in (INT32, INT64, FP32) or len(n) not in (2, 3) or n[0] < rope.n_axes or n[-1] != L or \
            (len(n) == 3 and n[1] != B) or positions.get_device() != dev:
        raise ValueError(f"positions must be int32, int64 or fp32 [axes, L] or [axes, B, L] on q's device with at "
                         f"least {rope.n_axes} axes")
    if q_out is not None or k_out is not None:
        for name, t, src in (("q_out", q_out, q), ("k_out", k_out, k)):
            if t is not None and (src is None or t.dtype is not dtype or t.shape != src.shape or
                                  t.get_device() != dev or (t.stride(3) != 1 and d != 1) or
                                  any(m > 1 and s == 0 for m, s in zip(t.shape, t.stride()))):
                raise ValueError(f"{name} must have its input's type and shape, contiguous columns and no shared rows")

    def call(ptr):
        if q_out is None:  # new and contiguous
            qo = q.new_empty((B, H, L, d))
            e, f, g = H * L * d, L * d, d
        else:
            qo = q_out
            e, f, g, _ = qo.stride()
        ko = kp = kop = None
        r, s, t, u, v, w = 0, 0, 0, 0, 0, 0
        if ks is not None:
            r, s, t, _ = ks
            if k_out is None:
                ko = k.new_empty((B, Hk, L, d))
                u, v, w = Hk * L * d, L * d, d
            else:
                ko = k_out
                u, v, w, _ = ko.stride()
            kp, kop = k.data_ptr(), ko.data_ptr()
        code = lib.bsa_rope_apply(q.data_ptr(), qo.data_ptr(), H, kp, kop, Hk, B, L, d, ty,
                                  _pack12(sb, sh, sl, e, f, g, r, s, t, u, v, w), positions.data_ptr(), pt,
                                  _pack3(ps[0], ps[1] if len(n) == 3 else 0, ps[-1]), rope._h, inverse, ptr)
        if code:
            _check(code, "bsa_rope_apply")
        return qo, ko
    return _on(dev, stream, call)


# ---------------------------------------------------------------- norms and residual of a block
def _vector_of(name, t, pt, C, dev):
    """Refuses a parameter that is not a vector [C] of type pt on device dev; its address."""
    if t.dtype is not pt or t.dim() != 1 or t.numel() != C or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [C] on x's device, of one type with the other parameters")
    return t.data_ptr()


def _norm_args(x, y, post, post_weight, post_bias, gate, branch_scale, stream_scale, pre, pre_weight, pre_bias, eps):
    """(the C structure, rows, device index)"""
    dtype, dev, shape, n = x.dtype, x.get_device(), x.shape, x.dim()
    ty = _type_of(dtype)
    if ty is None or ty > FP32 or dev < 0 or not x.is_contiguous() or n < 1 or shape[-1] < 1:
        raise ValueError("x must be a contiguous bf16, fp16 or fp32 CUDA tensor [.., C]")
    C = shape[-1]
    B = shape[0] if n > 1 else 1
    if post not in NORMS or pre not in NORMS:
        raise ValueError('post and pre must be "rms", "layer" or None')
    if y is None:
        if post is not None or gate is not None or pre is None or branch_scale != 1.0 or stream_scale != 1.0:
            raise ValueError("without y there is the pre norm alone")
    elif y.dtype is not dtype or y.shape != shape or y.get_device() != dev or not y.is_contiguous():
        raise ValueError("y must be like x")
    if (post is None and (post_weight is not None or post_bias is not None)) or \
            (pre is None and (pre_weight is not None or pre_bias is not None)):
        raise ValueError("a weight or bias needs its norm")
    pt = dtype
    for t in (post_weight, pre_weight, gate, post_bias, pre_bias):
        if t is not None:
            pt = t.dtype
            break
    pty = ty if pt is dtype else _type_of(pt)
    if pty != ty and pty != FP32:
        raise ValueError("parameters and gate must be all of x's type or all fp32")
    g, gate_rows = None, 1
    if gate is not None:
        if gate.dim() == 2 and gate.shape[0] in (1, B) and gate.shape[1] == C:
            if gate.dtype is not pt or gate.get_device() != dev or not gate.is_contiguous():
                raise ValueError("gate must be contiguous, on x's device and of one type with the parameters")
            g, gate_rows = gate.data_ptr(), gate.shape[0]
        else:
            g = _vector_of("gate (or [B, C])", gate, pt, C, dev)
    rows = x.numel() // C
    if rows > INT_MOST or C > INT_MOST:
        raise ValueError(_TOO_LARGE)
    a = BlockNormArgs(
        B, rows // B if B else 0, C, ty, pty, NORMS[post], NORMS[pre],
        None if post_weight is None else _vector_of("post_weight", post_weight, pt, C, dev),
        None if post_bias is None else _vector_of("post_bias", post_bias, pt, C, dev), g,
        None if pre_weight is None else _vector_of("pre_weight", pre_weight, pt, C, dev),
        None if pre_bias is None else _vector_of("pre_bias", pre_bias, pt, C, dev), gate_rows,
        branch_scale, stream_scale, eps)
    return a, rows, dev


def bsa_block_norm(x, y=None, post: Optional[str] = None, post_weight=None, post_bias=None, gate=None,
                   branch_scale: float = 1.0, stream_scale: float = 1.0, pre: Optional[str] = "rms",
                   pre_weight=None, pre_bias=None, eps: float = 1e-6, save_stats: bool = False, out=None,
                   normed=None, stream=None):
    """(stream, normed, stats) of the residual after a block and the norm before the next.

        stream = stream_scale x + branch_scale gate (N_post(y) post_weight + post_bias)
        normed = N_pre(stream) pre_weight + pre_bias

    x, y: contiguous bf16, fp16 or fp32 CUDA tensors [.., C], C <= 8192.  post, pre: "rms",
    "layer" or None for no norm (then normed is None).  gate: [C], or [B, C] with one row for
    each index of x's first axis (made for batch elements of many rows: the backward's time and
    workspace grow with the gate's rows).  Parameters and gate are all of x's type or all fp32; None
    stands for 1 (weights, gate) and 0 (biases).  Without y the stream is x itself and only
    the pre norm is taken.  stats (with ``save_stats``): fp32 [rows, 4], for the backward.
    out and normed may be given; they may be x or y, not each other.
    """
    import torch
    a, rows, dev = _norm_args(x, y, post, post_weight, post_bias, gate, branch_scale, stream_scale, pre, pre_weight,
                              pre_bias, eps)
    if out is not None or normed is not None:
        for name, t in (("out", out), ("normed", normed)):
            if t is not None and (t.shape != x.shape or t.dtype != x.dtype or not t.is_contiguous() or
                                  t.device != x.device):
                raise ValueError(f"{name} must be like x")
        if (out is not None and y is None) or (normed is not None and pre is None):
            raise ValueError("an output was given that the call does not have")

    def call(ptr):
        o = torch.empty_like(x) if y is not None and out is None else out
        n = torch.empty_like(x) if pre is not None and normed is None else normed
        st = x.new_empty((rows, 4), dtype=torch.float32) if save_stats else None
        code = lib.bsa_block_norm(a, x.data_ptr(), None if y is None else y.data_ptr(),
                                  None if o is None else o.data_ptr(), None if n is None else n.data_ptr(), _ptr(st),
                                  ptr)
        if code:
            _check(code, "bsa_block_norm")
        return (x if y is None else o), n, st
    return _on(dev, stream, call)


def bsa_block_norm_backward(dstream, dnormed, x, y, stats, post: Optional[str] = None, post_weight=None,
                            post_bias=None, gate=None, branch_scale: float = 1.0, stream_scale: float = 1.0,
                            pre: Optional[str] = "rms", pre_weight=None, pre_bias=None, params: bool = True,
                            stream=None):
    """Gradients of bsa_block_norm, as a dict with the keys x, y, post_weight, post_bias, gate,
    pre_weight and pre_bias (None for what the call does not have).

    dstream, dnormed: the loss's gradients by both results (None for zero).  x: the forward's
    stream, its first result.  y, stats and the other arguments: the forward's.  ``params``
    False leaves the parameters' and the gate's gradients out.
    """
    import torch
    a, rows, dev = _norm_args(x, y, post, post_weight, post_bias, gate, branch_scale, stream_scale, pre, pre_weight,
                              pre_bias, 0.0)
    shape, dtype = x.shape, x.dtype
    for name, t in (("dstream", dstream), ("dnormed", dnormed)):
        if t is not None and (t.shape != shape or t.dtype is not dtype or t.get_device() != dev or
                              not t.is_contiguous()):
            raise ValueError(f"{name} must be like x")
    if dnormed is not None and pre is None:
        raise ValueError("dnormed without a pre norm")
    if stats.dtype is not torch.float32 or stats.shape != (rows, 4) or stats.get_device() != dev or \
            not stats.is_contiguous():
        raise ValueError("stats must be the forward's fp32 [rows, 4]")

    def call(ptr):
        g = {"x": torch.empty_like(x), "y": None if y is None else torch.empty_like(y)}
        at = []  # addresses of the parameters' gradients
        for name, t in (("post_weight", post_weight), ("post_bias", post_bias), ("gate", gate),
                        ("pre_weight", pre_weight), ("pre_bias", pre_bias)):
            if params and t is not None:
                g[name] = t = torch.empty_like(t)
                at.append(t.data_ptr())
            else:
                g[name] = None
                at.append(None)
        ws, n = None, ctypes.c_size_t()
        if params and at != [None] * 5:
            code = lib.bsa_block_norm_backward_workspace_bytes(a, n)
            if code:
                _check(code, "bsa_block_norm_backward_workspace_bytes")
            ws = x.new_empty(n.value, dtype=torch.uint8)
        code = lib.bsa_block_norm_backward(a, _ptr(dstream), _ptr(dnormed), x.data_ptr(), _ptr(y), stats.data_ptr(),
                                           g["x"].data_ptr(), _ptr(g["y"]), *at, _ptr(ws), n.value, ptr)
        if code:
            _check(code, "bsa_block_norm_backward")
        return g
    return _on(dev, stream, call)


# ---------------------------------------------------------------- 8-bit floating point
def bsa_fp8_quantize(x, square: bool = False, rows: bool = True, cols: bool = False, dtype=None, stream=None):
    """8-bit codes of x [.., C] (R rows of C) with an fp32 scale for each block of 128.

    Returns (codes [R, C], scale [R, C/128]) with ``rows``: a block is 128 columns of one row;
    then (codes_t [C, R], scale_t [C, R/128]) with ``cols``: the same of x transposed.  With
    ``square`` blocks are 128 x 128 and the scales [R/128, C/128] and its transpose (sizes
    over 128 round up).  x: contiguous bf16, fp16 or fp32.  dtype: torch.float8_e4m3fn (the
    default) or torch.float8_e5m2.  Rows of codes start at multiples of 16 bytes.
    """
    import torch
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    ty, ct, dev = _type_of(x.dtype), _type_of(dtype), x.get_device()
    if ty is None or ty > FP32 or dev < 0 or not x.is_contiguous() or x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be a contiguous bf16, fp16 or fp32 CUDA tensor [.., C]")
    if ct != E4M3 and ct != E5M2:
        raise ValueError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2")
    if not rows and not cols:
        raise ValueError("ask for rows, cols or both")
    C = x.shape[-1]
    R = x.numel() // C
    if R > INT_MOST or C > INT_MOST:
        raise ValueError(_TOO_LARGE)

    def form(n, m):  # codes [n, m] in padded rows, their pitch, and their scales
        ld = (m + 15) // 16 * 16
        codes = x.new_empty((n, ld), dtype=dtype)
        scale = x.new_empty(((n + 127) // 128 if square else n, (m + 127) // 128), dtype=torch.float32)
        return (codes if ld == m else codes.narrow(1, 0, m)), scale, ld

    def call(ptr):
        codes, scale, ld = form(R, C) if rows else (None, None, 0)
        codes_t, scale_t, ld_t = form(C, R) if cols else (None, None, 0)
        code = lib.bsa_fp8_quantize(x.data_ptr(), ty, R, C, square, ct, _ptr(codes), ld, _ptr(scale), _ptr(codes_t),
                                    ld_t, _ptr(scale_t), ptr)
        if code:
            _check(code, "bsa_fp8_quantize")
        return (codes, scale, codes_t, scale_t) if rows and cols else (codes, scale) if rows else (codes_t, scale_t)
    return _on(dev, stream, call)


def _codes_pitch(name, t, ty, dev) -> int:
    """Refuses what is no matrix of 8-bit codes; the distance of its rows."""
    if (ty != E4M3 and ty != E5M2) or t.dim() != 2 or t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be an 8-bit CUDA matrix")
    ld, one = t.stride()
    n = t.shape[1]
    if n < 1 or (one != 1 and n > 1) or ld % 16 or ld < n or t.data_ptr() % 16:
        raise ValueError(f"{name} must have contiguous columns and rows starting at multiples of 16 bytes")
    return ld


def _scale_rows(name, scale, rows, kb, dev) -> int:
    """How many rows share a scale: 1 or 128."""
    if _type_of(scale.dtype) != FP32 or scale.dim() != 2 or not scale.is_contiguous() or scale.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous fp32 matrix on the codes' device")
    n, m = scale.shape
    if m == kb:
        if n == rows:
            return 1
        if n == (rows + 127) // 128:
            return 128
    raise ValueError(f"{name} must have a row for each row, or for each 128 rows, of its matrix, and a column for "
                     "each 128 of K")


def bsa_fp8_matmul_workspace_bytes(M: int, N: int, K: int) -> int:
    if (M | N | K) > INT_MOST:
        raise ValueError(_TOO_LARGE)
    n = ctypes.c_size_t()
    _check(lib.bsa_fp8_matmul_workspace_bytes(M, N, K, ctypes.byref(n)), "bsa_fp8_matmul_workspace_bytes")
    return n.value


def bsa_fp8_matmul(a, a_scale, b, b_scale, bias=None, out_dtype=None, out=None, workspace=None, stream=None):
    """a b^T [M, N] of 8-bit a [M, K] and b [N, K] with their scales, plus bias [N].

    a, b: torch.float8_e4m3fn or float8_e5m2, rows starting at multiples of 16 bytes (as
    bsa_fp8_quantize lays them out).  Scales: fp32 [rows, K/128] or [rows/128, K/128] (sizes
    over 128 round up).  bias: bf16 or fp32.  Result: bf16, or ``out_dtype`` fp32, or ``out``.
    workspace: uint8, at least bsa_fp8_matmul_workspace_bytes(M, N, K) bytes; allocated when
    omitted.
    """
    import torch
    at, bt, dev = _type_of(a.dtype), _type_of(b.dtype), a.get_device()
    lda, ldb = _codes_pitch("a", a, at, dev), _codes_pitch("b", b, bt, dev)
    (M, K), (N, Kb) = a.shape, b.shape
    if Kb != K:
        raise ValueError("a and b must have the same number of columns")
    if (M | N | K) > INT_MOST:
        raise ValueError(_TOO_LARGE)
    kb = (K + 127) // 128
    ar, br = _scale_rows("a_scale", a_scale, M, kb, dev), _scale_rows("b_scale", b_scale, N, kb, dev)
    bp, bty = None, BF16
    if bias is not None:
        bty = _type_of(bias.dtype)
        if bty not in (BF16, FP32) or bias.dim() != 1 or bias.numel() != N or not bias.is_contiguous() or \
                bias.get_device() != dev:
            raise ValueError("bias must be a contiguous bf16 or fp32 vector [N]")
        bp = bias.data_ptr()
    if out is not None:
        if out_dtype not in (None, out.dtype) or tuple(out.shape) != (M, N) or not out.is_contiguous() or \
                out.get_device() != dev:
            raise ValueError("out must be a contiguous tensor [M, N] of the result's type")
        out_dtype = out.dtype
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    ot = _type_of(out_dtype)
    if ot != BF16 and ot != FP32:
        raise ValueError("the result is bf16 or fp32")
    if workspace is not None and workspace.get_device() != dev:
        raise ValueError("workspace must be on a's device")

    def call(ptr):
        o = a_scale.new_empty((M, N), dtype=out_dtype) if out is None else out
        ws, n = workspace, 0
        if ws is not None:
            n = ws.numel() * ws.element_size()
        elif M > 8:  # fewer rows never split K
            n = bsa_fp8_matmul_workspace_bytes(M, N, K)
            ws = a_scale.new_empty(n, dtype=torch.uint8) if n else None
        code = lib.bsa_fp8_matmul(a.data_ptr(), at, lda, a_scale.data_ptr(), ar, b.data_ptr(), bt, ldb,
                                  b_scale.data_ptr(), br, bp, bty, M, N, K, o.data_ptr(), ot, _ptr(ws), n, ptr)
        if code:
            _check(code, "bsa_fp8_matmul")
        return o
    return _on(dev, stream, call)


def bsa_sync_status(stream=None) -> int:
    """Synchronises the stream; returns (and clears) the device status word."""
    return lib.bsa_sync_status(ctypes.c_void_p(_stream_ptr(stream)))


def bsa_debug_wait_timeout(timeout_ns: int, stream=None) -> None:
    _check(lib.bsa_debug_wait_timeout(ctypes.c_uint64(timeout_ns), ctypes.c_void_p(_stream_ptr(stream))),
           "bsa_debug_wait_timeout")


def bsa_debug_product_wait_timeout(timeout_ns: int, stream=None) -> None:
    _check(lib.bsa_debug_product_wait_timeout(ctypes.c_uint64(timeout_ns), ctypes.c_void_p(_stream_ptr(stream))),
           "bsa_debug_product_wait_timeout")


def header_symbols() -> list[str]:
    """Function names declared in include/bsa.h (parsed from the header text)."""
    import re
    hdr = os.path.join(os.path.dirname(os.path.dirname(_LIB_PATH)), "include", "bsa.h")
    with open(hdr) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:int|void|const char\*)\s+(bsa_\w+)\s*\(", text, re.M)))
