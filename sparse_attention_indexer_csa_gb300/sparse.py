"""ctypes binding of the operators that use the indexer's selection and of the
cache they read (the C ABI of ``include/csa_sparse.h``, exported by
``libcsa_index.so``): attention over listed blocks of keys, its gradients, the
same over a paged cache, and the norm and rotation of new tokens with their
append to that cache.

Argument marshalling only, as in ``attn.py``, whose rules for streams hold here.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import abi, attn
from .abi import _check
from .attn import NormRopeProblem, _Call, _check_norm_rope, _dtype, _ptr, _strides, _want

EXPORTED = (
    "csa_sparse_attn_forward",
    "csa_sparse_attn_backward",
    "csa_sparse_attn_workspace_size",
    "csa_norm_rope_append",
    "csa_sparse_abi_version",
)


class SparseProblem(ctypes.Structure):
    """Mirror of ``csa_sparse_problem`` (strides in elements; 0 = contiguous)."""

    _fields_ = [
        ("N", ctypes.c_int32), ("Tq", ctypes.c_int32), ("Tk", ctypes.c_int32), ("Hq", ctypes.c_int32),
        ("Hk", ctypes.c_int32), ("D", ctypes.c_int32), ("top_k", ctypes.c_int32), ("block", ctypes.c_int32),
        ("window", ctypes.c_int32), ("page", ctypes.c_int32), ("table_width", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
        ("idx_stride", ctypes.c_int64), ("table_stride", ctypes.c_int64),
        ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("k_stride_p", ctypes.c_int64), ("k_stride_t", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
        ("v_stride_p", ctypes.c_int64), ("v_stride_t", ctypes.c_int64), ("v_stride_h", ctypes.c_int64),
    ]


# The structures as packed bytes: half the time of their constructors, which a call of few tokens spends on the host.
_PACK_SPARSE = struct.Struct("=13if10q").pack
_PACK_NORM_ROPE = struct.Struct("=9if4q").pack
_PACK_APPEND = struct.Struct("=4i9q").pack


class AppendProblem(ctypes.Structure):
    """Mirror of ``csa_append_problem`` (strides in elements; 0 = contiguous)."""

    _fields_ = [
        ("N", ctypes.c_int32), ("pages", ctypes.c_int32), ("page", ctypes.c_int32), ("table_width", ctypes.c_int32),
        ("table_stride", ctypes.c_int64), ("v_stride_t", ctypes.c_int64), ("v_stride_h", ctypes.c_int64),
        ("kc_stride_p", ctypes.c_int64), ("kc_stride_t", ctypes.c_int64), ("kc_stride_h", ctypes.c_int64),
        ("vc_stride_p", ctypes.c_int64), ("vc_stride_t", ctypes.c_int64), ("vc_stride_h", ctypes.c_int64),
    ]


_ready = None


def load() -> ctypes.CDLL:
    """The library with this header's entry points typed (once)."""
    global _ready
    if _ready is not None:
        return _ready
    lib = attn.load()
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    S, R, A = ctypes.POINTER(SparseProblem), ctypes.POINTER(NormRopeProblem), ctypes.POINTER(AppendProblem)
    lib.csa_sparse_attn_forward.argtypes = [S] + [vp] * 11 + [sz, vp]
    lib.csa_sparse_attn_backward.argtypes = [S] + [vp] * 14 + [sz, vp]
    lib.csa_sparse_attn_workspace_size.argtypes = [S, i32]
    lib.csa_sparse_attn_workspace_size.restype = sz
    lib.csa_norm_rope_append.argtypes = [R, A] + [vp] * 14
    for name in ("csa_sparse_attn_forward", "csa_sparse_attn_backward", "csa_norm_rope_append",
                 "csa_sparse_abi_version"):
        getattr(lib, name).restype = i32
    _ready = lib
    return lib


# ----------------------------------------------------------------------------- argument checks
def _want_rows(t, what, rows, device):
    """An int32 matrix [rows, any] with contiguous rows (its stride is passed on)."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be [{rows}, any]")
    _want(t, what, (rows, t.shape[1]), torch.int32, device, True)
    if rows > 1 and t.shape[1] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"rows of {what} may not overlap")


def _row_stride(t):
    return 0 if t.shape[0] <= 1 else t.stride(0)


def _page_strides(t):
    """Page, token and head strides of [pages, page, H, D] (0 where the dimension has one entry)."""
    n, m, h, _ = t.shape
    a, b, c, _ = t.stride()
    return 0 if n <= 1 else a, 0 if m <= 1 else b, 0 if h <= 1 else c


def _check_pages(k_pages, v_pages, dtype, D, device):
    if k_pages.dim() != 4:
        raise ValueError("k_pages and v_pages must be [pages, page, Hk, D]")
    _want(k_pages, "k_pages", (*k_pages.shape[:3], D), dtype, device, True)
    _want(v_pages, "v_pages", k_pages.shape, dtype, device, True)
    if k_pages.shape[1] < 1:
        raise ValueError("a page holds one token at least")


# ----------------------------------------------------------------------------- attention over listed blocks
def make_sparse_problem(q, k, v, idx, cu_q, scale, block=1, window=0, causal=True, table=None) -> SparseProblem:
    """Problem of q [Tq,Hq,D], k and v [Tk,Hk,D] (or, with `table` [N,width],
    [pages,page,Hk,D]), idx [Tq,top_k] or None, and len(cu_q)-1 packed sequences;
    the tensors' strides are passed on."""
    Tq, Hq, D = q.shape
    top_k, idx_stride = (0, 0) if idx is None else (idx.shape[1], _row_stride(idx))
    if table is None:
        Tk, Hk, _ = k.shape
        page = width = table_stride = 0
        k_strides, v_strides = (0, *_strides(k)), (0, *_strides(v))
    else:
        pages, page, Hk, _ = k.shape
        Tk, width, table_stride = pages * page, table.shape[1], _row_stride(table)
        k_strides, v_strides = _page_strides(k), _page_strides(v)
    return SparseProblem.from_buffer_copy(_PACK_SPARSE(
        max(0, cu_q.numel() - 1), Tq, Tk, Hq, Hk, D, top_k, int(block), int(window), page, width, _dtype(q, "q"),
        1 if causal else 0, float(scale), idx_stride, table_stride, *_strides(q), *k_strides, *v_strides))


def sparse_attn_workspace_size(p: SparseProblem, which: int) -> int:
    return int(load().csa_sparse_attn_workspace_size(ctypes.byref(p), which))


def _check_sparse(q, idx, cu_q):
    if q.dim() != 3:
        raise ValueError("q must be [Tq, Hq, D]")
    dev = q.device
    _want(q, "q", q.shape, q.dtype, dev, True)
    if idx is not None:
        _want_rows(idx, "idx", q.shape[0], dev)
        if idx.shape[1] == 0:
            idx = None
    n = cu_q.numel()
    if n < 1:
        raise ValueError("cu_q holds one entry more than there are sequences")
    _want(cu_q, "cu_q", (n,), torch.int32, dev)
    return dev, n - 1, idx


def _check_packed(q, k, v, idx, cu_q, cu_k, k_len):
    dev, n, idx = _check_sparse(q, idx, cu_q)
    if k.dim() != 3:
        raise ValueError("k and v must be [Tk, Hk, D]")
    _want(k, "k", (k.shape[0], k.shape[1], q.shape[2]), q.dtype, dev, True)
    _want(v, "v", k.shape, q.dtype, dev, True)
    _want(cu_k, "cu_k", (n + 1,), torch.int32, dev)
    if k_len is not None:
        _want(k_len, "k_len", (n,), torch.int32, dev)
    return dev, idx


def _forward(p, dev, q, k, v, idx, cu_q, cu_k, k_len, table, workspace, stream):
    c = _Call(stream, dev, q, k, v, idx, cu_q, cu_k, k_len, table, workspace)
    try:
        out = c.new(q.shape, q.dtype)
        lse = c.new(q.shape[:2], torch.float32)
        if workspace is None:
            need = sparse_attn_workspace_size(p, 0)
            workspace = c.new((need,), torch.uint8) if need else None
        _check("csa_sparse_attn_forward", load().csa_sparse_attn_forward(
            ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(cu_q), _ptr(cu_k), _ptr(k_len), _ptr(table),
            _ptr(out), _ptr(lse), _ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(), c.handle))
    finally:
        c.done()
    return out, lse


def sparse_attn_forward(q, k, v, idx, cu_q, cu_k, scale, block=1, window=0, causal=True, k_len=None, workspace=None,
                        stream=None):
    """Attention of packed sequences over listed blocks: row t of q [Tq,Hq,D]
    attends to the keys of the blocks idx[t] (numbers of blocks of `block` keys
    within its sequence, -1: none; idx [Tq,top_k] int32, as index_fused writes
    them, or None) and to the last `window` keys up to its own position ->
    (out [Tq,Hq,D] in q's type, lse [Tq,Hq] fp32).  k and v [Tk,Hk,D] (views
    allowed), cu_q and cu_k [N+1] int32, k_len [N] int32 or None.  causal=False:
    all keys of the listed blocks, for entries whose visibility the selection has
    settled.  The outputs have no autograd history: gradients come from
    sparse_attn_backward."""
    dev, idx = _check_packed(q, k, v, idx, cu_q, cu_k, k_len)
    p = make_sparse_problem(q, k, v, idx, cu_q, scale, block, window, causal)
    return _forward(p, dev, q, k, v, idx, cu_q, cu_k, k_len, None, workspace, stream)


def sparse_attn_backward(dout, q, k, v, out, lse, idx, cu_q, cu_k, scale, block=1, window=0, causal=True, k_len=None,
                         workspace=None, stream=None):
    """Gradients of sparse_attn_forward for the cotangent dout of out
    (contiguous), from the forward's out and lse -> (dq, dk, dv), contiguous, in
    q's type.  With out and lse of several calls joined (lse by logaddexp, out by
    exp(lse_i - lse)), the gradients are this call's part of those of the joined out."""
    dev, idx = _check_packed(q, k, v, idx, cu_q, cu_k, k_len)
    _want(dout, "dout", q.shape, q.dtype, dev)
    _want(out, "out", q.shape, q.dtype, dev)
    _want(lse, "lse", q.shape[:2], torch.float32, dev)
    p = make_sparse_problem(q, k, v, idx, cu_q, scale, block, window, causal)
    c = _Call(stream, dev, dout, q, k, v, out, lse, idx, cu_q, cu_k, k_len, workspace)
    try:
        dq = c.new(q.shape, q.dtype)
        dk, dv = c.new(k.shape, k.dtype), c.new(v.shape, v.dtype)
        if workspace is None:
            workspace = c.new((sparse_attn_workspace_size(p, 1),), torch.uint8)
        _check("csa_sparse_attn_backward", load().csa_sparse_attn_backward(
            ctypes.byref(p), _ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(idx), _ptr(cu_q),
            _ptr(cu_k), _ptr(k_len), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
            workspace.numel() * workspace.element_size(), c.handle))
    finally:
        c.done()
    return dq, dk, dv


def sparse_attn_paged(q, k_pages, v_pages, table, idx, cu_q, k_len, scale, block=1, window=0, causal=True,
                      workspace=None, stream=None):
    """sparse_attn_forward over a paged cache: k_pages and v_pages
    [pages,page,Hk,D] (views allowed), table [N,width] int32 the pages of each
    sequence in order, k_len [N] int32 its cached tokens, the new ones among them
    -> (out, lse).  One query row per sequence is the decode step."""
    dev, n, idx = _check_sparse(q, idx, cu_q)
    _check_pages(k_pages, v_pages, q.dtype, q.shape[2], dev)
    _want_rows(table, "table", n, dev)
    _want(k_len, "k_len", (n,), torch.int32, dev)
    p = make_sparse_problem(q, k_pages, v_pages, idx, cu_q, scale, block, window, causal, table)
    return _forward(p, dev, q, k_pages, v_pages, idx, cu_q, None, k_len, table, workspace, stream)


# ----------------------------------------------------------------------------- append to a paged cache
def norm_rope_append(q, k, v, q_weight, k_weight, positions, freqs, cu_q, k_len, k_pages, v_pages, table, eps=1e-6,
                     rot_offset=0, interleaved=False, stream=None):
    """norm_rope of the new tokens' q [T,Hq,D] and k [T,Hk,D] (views allowed),
    with k's result and the values v [T,Hk,D] put into k_pages and v_pages
    [pages,page,Hk,D] (views allowed; changed in place) -> q_out [T,Hq,D].  Token
    cu_q[i] + r of sequence i, which has lq new tokens and k_len[i] tokens with
    them, takes the place k_len[i] - lq + r of the pages table[i] (table [N,width]
    int32; cu_q [N+1], k_len [N] int32).  A token whose place has no valid page is
    not stored, and device_status() reports it."""
    if k is None or v is None:
        raise ValueError("k and v are needed")
    dev = _check_norm_rope(q, k, q_weight, k_weight, positions, freqs)
    _want(v, "v", k.shape, q.dtype, dev, True)
    n = cu_q.numel() - 1
    if n < 0:
        raise ValueError("cu_q holds one entry more than there are sequences")
    _want(cu_q, "cu_q", (n + 1,), torch.int32, dev)
    _want(k_len, "k_len", (n,), torch.int32, dev)
    _check_pages(k_pages, v_pages, q.dtype, q.shape[2], dev)
    if k_pages.shape[2] != k.shape[1]:
        raise ValueError(f"k_pages holds {k_pages.shape[2]} heads, k {k.shape[1]}")
    _want_rows(table, "table", n, dev)
    T, Hq, D = q.shape
    p = NormRopeProblem.from_buffer_copy(_PACK_NORM_ROPE(
        T, Hq, k.shape[1], D, 2 * freqs.numel(), int(rot_offset), 1 if interleaved else 0, _dtype(q, "q"),
        _dtype(q_weight, "q_weight"), float(eps), *_strides(q), *_strides(k)))
    a = AppendProblem.from_buffer_copy(_PACK_APPEND(
        n, k_pages.shape[0], k_pages.shape[1], table.shape[1], _row_stride(table), *_strides(v),
        *_page_strides(k_pages), *_page_strides(v_pages)))
    c = _Call(stream, dev, q, k, v, q_weight, k_weight, positions, freqs, cu_q, k_len, k_pages, v_pages, table)
    try:
        q_out = c.new(q.shape, q.dtype)
        _check("csa_norm_rope_append", load().csa_norm_rope_append(
            ctypes.byref(p), ctypes.byref(a), _ptr(q), _ptr(k), _ptr(v), _ptr(q_weight), _ptr(k_weight),
            _ptr(positions), _ptr(freqs), _ptr(cu_q), _ptr(k_len), _ptr(table), _ptr(q_out), _ptr(k_pages),
            _ptr(v_pages), c.handle))
    finally:
        c.done()
    return q_out
