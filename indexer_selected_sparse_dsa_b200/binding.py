"""ctypes binding of libdsa (include/dsa.h): argument marshalling only.

Every function here takes torch tensors that already live on the current CUDA
device, checks dtypes and shapes, and passes raw pointers and sizes to the C
entry point of the same name.  All arithmetic happens in the CUDA kernels.
There is no fallback: if ``libdsa.so`` is missing or fails to load, every
call raises.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libdsa.so")

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_WORKSPACE, DSA_ERR_CUDA, DSA_ERR_TIMEOUT, DSA_ERR_UNSUPPORTED, DSA_ERR_BAD_ROW = range(7)
(DSA_OP_INDEXER, DSA_OP_TOPK, DSA_OP_SPARSE_MLA, DSA_OP_FORWARD, DSA_OP_INDEXER_TOPK, DSA_OP_DENSE_SPARSE,
 DSA_OP_BLOCK_SPARSE, DSA_OP_PAGED_MLA) = range(8)
BLOCK_TOPK = 16
INDEX_HEADS, INDEX_DIM, HEADS, LATENT, ROPE, ROW, MAX_TOPK = 32, 128, 64, 512, 64, 576, 2048
NOALLOC_MAX_ROWS = 8192
ROW8 = 640

_STATUS_NAMES = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_WORKSPACE", 3: "DSA_ERR_CUDA",
                 4: "DSA_ERR_TIMEOUT", 5: "DSA_ERR_UNSUPPORTED", 6: "DSA_ERR_BAD_ROW"}


class DSAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


_lib = None


def lib():
    """Load libdsa.so (built in-tree).  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdsa.so not built ({LIB_PATH}); run python -m indexer_selected_sparse_dsa_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        L.dsa_workspace_size.argtypes = [I, I, I64, I]
        L.dsa_workspace_size.restype = SZ
        L.dsa_indexer_scores.argtypes = [P, P, P, I64, P, P, I, P, I64, P, SZ, P]
        L.dsa_topk.argtypes = [P, I64, P, I, I, P, P]
        L.dsa_sparse_mla_attn.argtypes = [P, P, I64, P, P, I, I, F, P, P, P, SZ, P]
        L.dsa_forward.argtypes = [P, P, P, P, P, I64, P, P, I, I64, I, F, P, P, P, P, SZ, P]
        L.dsa_sync_status.argtypes = [P]
        L.dsa_indexer_topk.argtypes = [P, P, P, I64, P, P, I, I64, I, P, P, SZ, P]
        L.dsa_indexer_topk.restype = I
        L.dsa_indexer_scores_noalloc.argtypes = [P, P, P, I64, P, P, I, P, I64, P]
        L.dsa_dense_sparse_attn.argtypes = [P, P, I64, P, P, P, I, I, I, P, F, P, P, P, P, SZ, P]
        L.dsa_dense_sparse_attn.restype = I
        L.dsa_indexer_scores_noalloc.restype = I
        L.dsa_block_sparse_attn.argtypes = [P, P, P, P, P, I64, P, P, I, I64, P, F, P, P, P, P, SZ, P]
        L.dsa_block_sparse_attn.restype = I
        paged = [P, P, P, I, I]             # cu_q, seq_len, page_table, batch, max_pages
        cache = [P, P, I, I]                # kv8, kv_scale, n_pages, page_size
        L.dsa_cache_write.argtypes = [P, I64, I, *paged, *cache, P]
        L.dsa_cache_read.argtypes = [*cache, P, P, I, I, P, P, I64, P]
        L.dsa_paged_mla_attn.argtypes = [P, I, *paged, *cache, F, P, P, P, SZ, P]
        L.dsa_paged_sparse_mla_attn.argtypes = [P, I, *paged, P, I, *cache, F, P, P, P, SZ, P]
        for name in ("dsa_cache_write", "dsa_cache_read", "dsa_paged_mla_attn", "dsa_paged_sparse_mla_attn"):
            getattr(L, name).restype = I
        L.dsa_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        L.dsa_set_wait_limit_ns.restype = None
        L.dsa_check_wait_timeout.argtypes = [P]
        L.dsa_check_wait_timeout.restype = I
        L.dsa_last_error_string.restype = ctypes.c_char_p
        L.dsa_abi_version.restype = I
        for name in ("dsa_indexer_scores", "dsa_topk", "dsa_sparse_mla_attn", "dsa_forward", "dsa_sync_status"):
            getattr(L, name).restype = I
        _lib = L
    return _lib


def last_error() -> str:
    return lib().dsa_last_error_string().decode()


def _check(rc: int):
    if rc != DSA_OK:
        raise DSAError(rc, last_error())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, dtype, shape=None, name=""):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def dsa_workspace_size(op: int, T: int, max_n_vis: int, topk: int) -> int:
    return int(lib().dsa_workspace_size(op, T, max_n_vis, topk))


def dsa_indexer_scores(q_I, w, k_I, kv_start, n_vis, scores, ws, stream=None):
    import torch
    T = n_vis.shape[0]
    _need(q_I, torch.bfloat16, (T, INDEX_HEADS, INDEX_DIM), "q_I")
    _need(w, torch.bfloat16, (T, INDEX_HEADS), "w")
    _need(k_I, torch.bfloat16, None, "k_I")
    _need(kv_start, torch.int64, (T,), "kv_start")
    _need(n_vis, torch.int32, (T,), "n_vis")
    _need(scores, torch.float32, None, "scores")
    _need(ws, torch.uint8, None, "ws")
    _check(lib().dsa_indexer_scores(_ptr(q_I), _ptr(w), _ptr(k_I), k_I.shape[0], _ptr(kv_start), _ptr(n_vis), T,
                                    _ptr(scores), scores.shape[1], _ptr(ws), ws.numel(), _stream(stream)))


def dsa_indexer_scores_noalloc(q_I, w, k_I, kv_start, n_vis, scores, stream=None):
    """dsa_indexer_scores for callers that cannot allocate: no workspace; the
    library keeps the plan in its own fixed device array (at most
    NOALLOC_MAX_ROWS rows; calls must not overlap on the GPU)."""
    import torch
    T = n_vis.shape[0]
    _need(q_I, torch.bfloat16, (T, INDEX_HEADS, INDEX_DIM), "q_I")
    _need(w, torch.bfloat16, (T, INDEX_HEADS), "w")
    _need(k_I, torch.bfloat16, None, "k_I")
    _need(kv_start, torch.int64, (T,), "kv_start")
    _need(n_vis, torch.int32, (T,), "n_vis")
    _need(scores, torch.float32, None, "scores")
    _check(lib().dsa_indexer_scores_noalloc(_ptr(q_I), _ptr(w), _ptr(k_I), k_I.shape[0], _ptr(kv_start),
                                            _ptr(n_vis), T, _ptr(scores), scores.shape[1], _stream(stream)))


def dsa_indexer_topk(q_I, w, k_I, kv_start, n_vis, max_n_vis, topk, idx, ws, stream=None):
    import torch
    T = n_vis.shape[0]
    _need(q_I, torch.bfloat16, (T, INDEX_HEADS, INDEX_DIM), "q_I")
    _need(w, torch.bfloat16, (T, INDEX_HEADS), "w")
    _need(k_I, torch.bfloat16, None, "k_I")
    _need(kv_start, torch.int64, (T,), "kv_start")
    _need(n_vis, torch.int32, (T,), "n_vis")
    _need(idx, torch.int32, (T, topk), "idx")
    _need(ws, torch.uint8, None, "ws")
    _check(lib().dsa_indexer_topk(_ptr(q_I), _ptr(w), _ptr(k_I), k_I.shape[0], _ptr(kv_start), _ptr(n_vis), T,
                                  int(max_n_vis), topk, _ptr(idx), _ptr(ws), ws.numel(), _stream(stream)))


def dsa_topk(scores, n_vis, topk, idx, stream=None):
    import torch
    T = n_vis.shape[0]
    _need(scores, torch.float32, None, "scores")
    _need(n_vis, torch.int32, (T,), "n_vis")
    _need(idx, torch.int32, (T, topk), "idx")
    _check(lib().dsa_topk(_ptr(scores), scores.shape[1], _ptr(n_vis), T, topk, _ptr(idx), _stream(stream)))


def dsa_sparse_mla_attn(q, kv, kv_start, idx, scale, o_lat, lse=None, ws=None, stream=None):
    import torch
    T, topk = idx.shape
    _need(q, torch.bfloat16, (T, HEADS, ROW), "q")
    _need(kv, torch.bfloat16, None, "kv")
    _need(kv_start, torch.int64, (T,), "kv_start")
    _need(idx, torch.int32, (T, topk), "idx")
    _need(o_lat, torch.float32, (T, HEADS, LATENT), "o_lat")
    if lse is not None:
        _need(lse, torch.float32, (T, HEADS), "lse")
    if ws is not None:
        _need(ws, torch.uint8, None, "ws")
    _check(lib().dsa_sparse_mla_attn(_ptr(q), _ptr(kv), kv.shape[0], _ptr(kv_start), _ptr(idx), T, topk,
                                     float(scale), _ptr(o_lat), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(),
                                     _stream(stream)))


def dsa_dense_sparse_attn(q, kv, kv_start, n_vis, idx, window, gate, scale, o_lat, lse_dense=None, lse_sparse=None,
                          ws=None, stream=None):
    import torch
    T, topk = idx.shape
    _need(q, torch.bfloat16, (T, HEADS, ROW), "q")
    _need(kv, torch.bfloat16, None, "kv")
    _need(kv_start, torch.int64, (T,), "kv_start")
    _need(n_vis, torch.int32, (T,), "n_vis")
    _need(idx, torch.int32, (T, topk), "idx")
    _need(gate, torch.float32, (T, HEADS), "gate")
    _need(o_lat, torch.float32, (T, HEADS, LATENT), "o_lat")
    for t, nm in ((lse_dense, "lse_dense"), (lse_sparse, "lse_sparse")):
        if t is not None:
            _need(t, torch.float32, (T, HEADS), nm)
    if ws is not None:
        _need(ws, torch.uint8, None, "ws")
    _check(lib().dsa_dense_sparse_attn(_ptr(q), _ptr(kv), kv.shape[0], _ptr(kv_start), _ptr(n_vis), _ptr(idx), T, topk,
                                       int(window), _ptr(gate), float(scale), _ptr(o_lat), _ptr(lse_dense),
                                       _ptr(lse_sparse), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def dsa_forward(q_I, w, k_I, q, kv, kv_start, n_vis, max_n_vis, topk, scale, o_lat, lse, idx_out, ws, stream=None):
    import torch
    T = n_vis.shape[0]
    _need(q_I, torch.bfloat16, (T, INDEX_HEADS, INDEX_DIM), "q_I")
    _need(w, torch.bfloat16, (T, INDEX_HEADS), "w")
    _need(k_I, torch.bfloat16, None, "k_I")
    _need(q, torch.bfloat16, (T, HEADS, ROW), "q")
    _need(kv, torch.bfloat16, None, "kv")
    if k_I.shape[0] != kv.shape[0]:
        raise ValueError("k_I and kv must have the same number of cache rows")
    _need(kv_start, torch.int64, (T,), "kv_start")
    _need(n_vis, torch.int32, (T,), "n_vis")
    _need(o_lat, torch.float32, (T, HEADS, LATENT), "o_lat")
    if lse is not None:
        _need(lse, torch.float32, (T, HEADS), "lse")
    if idx_out is not None:
        _need(idx_out, torch.int32, (T, topk), "idx_out")
    _need(ws, torch.uint8, None, "ws")
    _check(lib().dsa_forward(_ptr(q_I), _ptr(w), _ptr(k_I), _ptr(q), _ptr(kv), kv.shape[0], _ptr(kv_start),
                             _ptr(n_vis), T, int(max_n_vis), topk, float(scale), _ptr(o_lat), _ptr(lse),
                             _ptr(idx_out), _ptr(ws), ws.numel(), _stream(stream)))


def dsa_block_sparse_attn(q_I, w, k_I, q, kv, kv_start, n_vis, max_n_vis, gates, scale, o_lat, lse, blocks_out, ws,
                          stream=None):
    """Block-level variant: local / anchor / top-16-block branches fused with
    gates [T, 64, 3]; lse [3, T, 64] and blocks_out [T, 16] may be None."""
    import torch
    T = n_vis.shape[0]
    for t_, nm in ((q_I, "q_I"), (w, "w"), (k_I, "k_I"), (q, "q"), (kv, "kv")):
        _need(t_, torch.bfloat16, None, nm)
    _need(q_I, torch.bfloat16, (T, INDEX_HEADS, INDEX_DIM), "q_I")
    _need(q, torch.bfloat16, (T, HEADS, ROW), "q")
    _need(kv, torch.bfloat16, (kv.shape[0], ROW), "kv")
    _need(k_I, torch.bfloat16, (kv.shape[0], INDEX_DIM), "k_I")
    _need(kv_start, torch.int64, (T,), "kv_start")
    _need(n_vis, torch.int32, (T,), "n_vis")
    _need(gates, torch.float32, (T, HEADS, 3), "gates")
    _need(o_lat, torch.float32, (T, HEADS, LATENT), "o_lat")
    if lse is not None:
        _need(lse, torch.float32, (3, T, HEADS), "lse")
    if blocks_out is not None:
        _need(blocks_out, torch.int32, (T, BLOCK_TOPK), "blocks_out")
    _need(ws, torch.uint8, None, "ws")
    _check(lib().dsa_block_sparse_attn(_ptr(q_I), _ptr(w), _ptr(k_I), _ptr(q), _ptr(kv), kv.shape[0], _ptr(kv_start),
                                       _ptr(n_vis), T, int(max_n_vis), _ptr(gates), float(scale), _ptr(o_lat),
                                       _ptr(lse), _ptr(blocks_out), _ptr(ws), ws.numel(), _stream(stream)))


# A decode step calls the paged entry points once per layer, so their checks are made for few Python calls: one pass
# over (tensor, dtype, shape, name) with the common case tested in place, and plain integers to ctypes.

def _device():
    """The current device; None before there is any CUDA tensor (and so none to check)."""
    import torch
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else None


def _check_all(dev, *specs):
    """Check each (tensor, dtype, shape, name); None for an optional tensor.  Returns the addresses.

    The kernels run on the current device `dev`: a tensor of another one would be a wild pointer to them."""
    ptrs = []
    for t, dtype, shape, name in specs:
        if t is None:
            ptrs.append(None)
            continue
        try:
            good = t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous()
        except AttributeError:
            good = False
        if not good:
            _need(t, dtype, shape, name)
            raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")
        ptrs.append(t.data_ptr())
    return ptrs


def _raw_stream(stream, dev):
    import torch
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _rows(t, name):
    """Length of a tensor's first dimension; what has none is found here, everything else by _check_all."""
    try:
        return t.shape[0]
    except (AttributeError, IndexError, TypeError):
        raise TypeError(f"{name} must be a CUDA tensor of at least one dimension") from None


def _paged_sizes(seq_len, page_table, kv8):
    """(batch, max_pages, n_pages, page_size); a wrong number of dimensions is found here, wrong sizes by _check_all."""
    try:
        (batch,), (_, max_pages), (n_pages, page_size, _) = seq_len.shape, page_table.shape, kv8.shape
    except (AttributeError, TypeError, ValueError):
        for t, nd, name in ((seq_len, 1, "seq_len"), (page_table, 2, "page_table"), (kv8, 3, "kv8")):
            if getattr(t, "ndim", None) != nd:
                raise TypeError(f"{name} must be a tensor of {nd} dimension{'s' if nd > 1 else ''}") from None
        raise
    return batch, max_pages, n_pages, page_size


def dsa_cache_write(rows, cu_q, seq_len, page_table, kv8, kv_scale, stream=None):
    """Quantise latent rows [T, 576] bf16 (their row stride is free, the rest contiguous)
    into the paged cache kv8 [n_pages, page_size, 640] uint8, kv_scale [n_pages, page_size]."""
    import torch
    batch, max_pages, n_pages, page_size = _paged_sizes(seq_len, page_table, kv8)
    i32, dev = torch.int32, _device()
    cu, sl, pt, k8, ks = _check_all(
        dev, (cu_q, i32, (batch + 1,), "cu_q"), (seq_len, i32, (batch,), "seq_len"),
        (page_table, i32, (batch, max_pages), "page_table"), (kv8, torch.uint8, (n_pages, page_size, ROW8), "kv8"),
        (kv_scale, torch.float32, (n_pages, page_size), "kv_scale"))
    if not isinstance(rows, torch.Tensor) or not rows.is_cuda or rows.dtype != torch.bfloat16:
        raise TypeError("rows must be a CUDA tensor of torch.bfloat16")
    if rows.ndim != 2 or rows.shape[1] != ROW or rows.stride(1) != 1:
        raise ValueError(f"rows must have shape (T, {ROW}) with contiguous rows, got {tuple(rows.shape)}, "
                         f"strides {rows.stride()}")
    if rows.get_device() != dev:
        raise ValueError(f"rows must be on the current device cuda:{dev}, got {rows.device}")
    T = rows.shape[0]
    _check(lib().dsa_cache_write(rows.data_ptr(), rows.stride(0) if T > 1 else ROW, T, cu, sl, pt, batch, max_pages, k8,
                                 ks, n_pages, page_size, _raw_stream(stream, dev)))


def dsa_cache_read(kv8, kv_scale, seq_len, page_table, kv_start, kv, stream=None):
    """Unpack every sequence of the paged cache to flat bf16 rows kv[kv_start[b] + s]."""
    import torch
    batch, max_pages, n_pages, page_size = _paged_sizes(seq_len, page_table, kv8)
    cache_rows = _rows(kv, "kv")
    i32, dev = torch.int32, _device()
    k8, ks, sl, pt, start, flat = _check_all(
        dev, (kv8, torch.uint8, (n_pages, page_size, ROW8), "kv8"),
        (kv_scale, torch.float32, (n_pages, page_size), "kv_scale"), (seq_len, i32, (batch,), "seq_len"),
        (page_table, i32, (batch, max_pages), "page_table"), (kv_start, torch.int64, (batch,), "kv_start"),
        (kv, torch.bfloat16, (cache_rows, ROW), "kv"))
    _check(lib().dsa_cache_read(k8, ks, n_pages, page_size, sl, pt, batch, max_pages, start, flat, cache_rows,
                                _raw_stream(stream, dev)))


def _paged_attn(name, q, cu_q, seq_len, page_table, idx, kv8, kv_scale, scale, o_lat, lse, ws, stream):
    import torch
    batch, max_pages, n_pages, page_size = _paged_sizes(seq_len, page_table, kv8)
    i32, f32, bf16, dev = torch.int32, torch.float32, torch.bfloat16, _device()
    T, ws_bytes = _rows(q, "q"), _rows(ws, "ws")
    if idx is not None and getattr(idx, "ndim", None) != 2:
        raise TypeError("idx must be a tensor of 2 dimensions")
    qp, cu, sl, pt, k8, ks, op, lp, wp = _check_all(
        dev, (q, bf16, (T, HEADS, ROW), "q"), (cu_q, i32, (batch + 1,), "cu_q"), (seq_len, i32, (batch,), "seq_len"),
        (page_table, i32, (batch, max_pages), "page_table"), (kv8, torch.uint8, (n_pages, page_size, ROW8), "kv8"),
        (kv_scale, f32, (n_pages, page_size), "kv_scale"), (o_lat, bf16, (T, HEADS, LATENT), "o_lat"),
        (lse, f32, (T, HEADS), "lse"), (ws, torch.uint8, (ws_bytes,), "ws"))
    sel = ()
    if idx is not None:
        sel = (*_check_all(dev, (idx, i32, (T, idx.shape[1]), "idx")), idx.shape[1])
    _check(getattr(lib(), name)(qp, T, cu, sl, pt, batch, max_pages, *sel, k8, ks, n_pages, page_size, scale, op, lp, wp,
                                ws_bytes, _raw_stream(stream, dev)))


def dsa_paged_mla_attn(q, cu_q, seq_len, page_table, kv8, kv_scale, scale, o_lat, lse, ws, stream=None):
    """Dense latent attention of the new tokens over their sequences' pages; o_lat is bf16, lse may be None."""
    _paged_attn("dsa_paged_mla_attn", q, cu_q, seq_len, page_table, None, kv8, kv_scale, scale, o_lat, lse, ws, stream)


def dsa_paged_sparse_mla_attn(q, cu_q, seq_len, page_table, idx, kv8, kv_scale, scale, o_lat, lse, ws, stream=None):
    """Latent attention of the new tokens over their selected positions idx [T, topk] of the paged cache."""
    if idx is None:
        raise TypeError("idx must be a CUDA tensor")
    _paged_attn("dsa_paged_sparse_mla_attn", q, cu_q, seq_len, page_table, idx, kv8, kv_scale, scale, o_lat, lse, ws,
                stream)


def dsa_sync_status(stream=None):
    _check(lib().dsa_sync_status(_stream(stream)))


def dsa_set_wait_limit_ns(ns: int):
    """Limit of every bounded device wait, in ns (0: the default)."""
    lib().dsa_set_wait_limit_ns(int(ns))


def dsa_check_wait_timeout(stream=None):
    """Enqueue the hang-protection probe (a wait nothing completes); the next
    dsa_sync_status reports DSA_ERR_TIMEOUT."""
    _check(lib().dsa_check_wait_timeout(_stream(stream)))


def workspace(op, T, max_n_vis, topk, device=None):
    """Allocate a workspace tensor (torch owns the memory; 256-byte aligned)."""
    import torch
    n = max(dsa_workspace_size(op, T, max_n_vis, topk), 256)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")
