"""ctypes binding of the operators around the indexer (the C ABI of
``include/csa_attn.h``, exported by ``libcsa_index.so``): the norm and rotation
of queries and keys, and causal attention over packed sequences.

Argument marshalling only, as in ``abi.py``.  Every helper takes ``stream``
(default: the current stream of the tensors' device); the tensors it takes and
those it allocates are recorded on that stream, so they may be dropped while its
work is in flight.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import abi
from .abi import CSA_BF16, CSA_F32, _check

CSA_F16 = 2

EXPORTED = (
    "csa_rope_freqs",
    "csa_norm_rope",
    "csa_norm_rope_backward",
    "csa_norm_rope_workspace_size",
    "csa_attn_forward",
    "csa_attn_backward",
    "csa_attn_workspace_size",
    "csa_attn_abi_version",
)

_DTYPES = {torch.bfloat16: CSA_BF16, torch.float32: CSA_F32, torch.float16: CSA_F16}


class NormRopeProblem(ctypes.Structure):
    """Mirror of ``csa_norm_rope_problem`` (strides in elements; 0 = contiguous)."""

    _fields_ = [
        ("T", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32), ("D", ctypes.c_int32),
        ("rot", ctypes.c_int32), ("rot_offset", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
        ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("k_stride_t", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
    ]


class AttnProblem(ctypes.Structure):
    """Mirror of ``csa_attn_problem`` (strides in elements; 0 = contiguous)."""

    _fields_ = [
        ("N", ctypes.c_int32), ("Tq", ctypes.c_int32), ("Tk", ctypes.c_int32), ("Hq", ctypes.c_int32),
        ("Hk", ctypes.c_int32), ("D", ctypes.c_int32), ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("k_stride_t", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
        ("v_stride_t", ctypes.c_int64), ("v_stride_h", ctypes.c_int64),
    ]


_ready = None


def load() -> ctypes.CDLL:
    """The library with this header's entry points typed (once)."""
    global _ready
    if _ready is not None:
        return _ready
    lib = abi.load()
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    R, A = ctypes.POINTER(NormRopeProblem), ctypes.POINTER(AttnProblem)
    lib.csa_rope_freqs.argtypes = [ctypes.c_double, i32, vp]
    lib.csa_norm_rope.argtypes = [R] + [vp] * 9
    lib.csa_norm_rope_backward.argtypes = [R] + [vp] * 13 + [sz, vp]
    lib.csa_norm_rope_workspace_size.argtypes = [R]
    lib.csa_norm_rope_workspace_size.restype = sz
    lib.csa_attn_forward.argtypes = [A] + [vp] * 9 + [sz, vp]
    lib.csa_attn_backward.argtypes = [A] + [vp] * 13 + [sz, vp]
    lib.csa_attn_workspace_size.argtypes = [A, i32]
    lib.csa_attn_workspace_size.restype = sz
    for name in ("csa_rope_freqs", "csa_norm_rope", "csa_norm_rope_backward", "csa_attn_forward",
                 "csa_attn_backward", "csa_attn_abi_version"):
        getattr(lib, name).restype = i32
    _ready = lib
    return lib


# ----------------------------------------------------------------------------- argument checks
def _dtype(t: torch.Tensor, what: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bf16, fp16 or fp32, not {t.dtype}")
    return code


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr() or None


def _want(t: torch.Tensor, what: str, shape, dtype, device, strided: bool = False):
    """Shape, type, device and layout of one argument."""
    if t.device != device or t.dtype != dtype or t.shape != shape or device.type != "cuda":
        if not t.is_cuda:
            raise ValueError(f"{what} must live on the GPU")
        if t.device != device:
            raise ValueError(f"{what} is on {t.device}, the call's tensors on {device}")
        if t.dtype != dtype:
            raise ValueError(f"{what} must be {dtype}, not {t.dtype}")
        raise ValueError(f"{what} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.is_contiguous():
        return
    if not strided:
        raise ValueError(f"{what} must be contiguous")
    st = t.stride()
    if t.numel() and shape[-1] != 1 and st[-1] != 1:
        raise ValueError(f"the innermost dimension of {what} must be contiguous")
    if any(n > 1 and x == 0 for n, x in zip(shape[:-1], st)):
        raise ValueError(f"{what} may not repeat memory (stride 0)")


def _current_stream(device) -> int:
    """Handle of the current stream (without the stream object where torch has a call for that)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None and device.index is not None:
        return raw(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class _Call:
    """Device and stream of one call: the stream as the library takes it, and
    the memory that the call uses and allocates."""

    __slots__ = ("device", "stream", "handle", "guard")

    def __init__(self, stream, device, *used):
        self.device = device
        # kernels go to the current device, so it has to be the tensors' one
        self.guard = None
        if device.index is not None and torch.cuda.current_device() != device.index:
            self.guard = torch.cuda.device(device)
            self.guard.__enter__()
        try:
            self._take(stream, used)
        except BaseException:
            self.done()  # a stream that is none leaves the current device as it was
            raise

    def _take(self, stream, used):
        device = self.device
        self.stream = None  # a stream other than the current one
        self.handle = _current_stream(device)
        if stream is not None:
            handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
            if handle != self.handle:
                self.stream = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(handle, device=device)
                # the allocator's memory may still be in use by work of the current stream
                self.stream.wait_stream(torch.cuda.current_stream(device))
                self.handle = handle
                for t in used:
                    if t is not None and t.numel():
                        t.record_stream(self.stream)

    def new(self, shape, dtype) -> torch.Tensor:
        """An uninitialised tensor; its memory is not given to other work
        before what the call's stream holds at its release has run."""
        t = torch.empty(shape, dtype=dtype, device=self.device)
        if self.stream is not None and t.numel():
            t.record_stream(self.stream)
        return t

    def done(self):
        if self.guard is not None:
            self.guard.__exit__(None, None, None)


def _strides(t: torch.Tensor):
    """Token and head strides (0 where the dimension has one entry)."""
    n, m = t.shape[0], t.shape[1]
    a, b, _ = t.stride()
    return 0 if n <= 1 else a, 0 if m <= 1 else b


# ----------------------------------------------------------------------------- norm + rotation
def rope_freqs(rot: int, theta: float = 10000.0, device=None) -> torch.Tensor:
    """Turns per position of the rot/2 pairs, theta^(-2i/rot)/(2 pi), as 64-bit
    fixed-point fractions: int64 [rot/2] (the bits of uint64) on `device`
    (default: the current GPU).  Made once and kept by the caller."""
    host = torch.empty(max(rot // 2, 0), dtype=torch.int64)
    _check("csa_rope_freqs", load().csa_rope_freqs(float(theta), int(rot), ctypes.c_void_p(host.data_ptr())))
    return host.to(torch.device("cuda", torch.cuda.current_device()) if device is None else device)


def make_norm_rope_problem(q, k, q_weight, freqs, eps=1e-6, rot_offset=0, interleaved=False) -> NormRopeProblem:
    """Problem of q [T,Hq,D] and k [T,Hk,D] (or None); their strides are passed on."""
    T, Hq, D = q.shape
    p = NormRopeProblem(T, Hq, 0 if k is None else k.shape[1], D, 2 * freqs.numel(), int(rot_offset),
                        1 if interleaved else 0, _dtype(q, "q"), _dtype(q_weight, "q_weight"), float(eps))
    p.q_stride_t, p.q_stride_h = _strides(q)
    if k is not None:
        p.k_stride_t, p.k_stride_h = _strides(k)
    return p


def _check_norm_rope(q, k, q_weight, k_weight, positions, freqs):
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, D]")
    if (k is None) != (k_weight is None):
        raise ValueError("k and k_weight come together")
    T, Hq, D = q.shape
    dev = q.device
    _want(q, "q", q.shape, q.dtype, dev, True)
    _want(q_weight, "q_weight", (D,), q_weight.dtype, dev)
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k must be [T, Hk, D]")
        _want(k, "k", (T, k.shape[1], D), q.dtype, dev, True)
        _want(k_weight, "k_weight", (D,), q_weight.dtype, dev)
    _want(positions, "positions", (T,), torch.int64, dev)
    _want(freqs, "freqs", (freqs.numel(),), torch.int64, dev)
    return dev


def norm_rope(q, k, q_weight, k_weight, positions, freqs, eps=1e-6, rot_offset=0, interleaved=False, stream=None):
    """Norm of every head of q [T,Hq,D] and k [T,Hk,D] with the weights [D], and
    the rotation of 2*len(freqs) of its values from rot_offset on, by
    positions [T] int64 -> (q_out, k_out), contiguous, in the inputs' type.
    k and k_weight may be None (k_out is None).  q and k may be views.  The
    outputs have no autograd history: gradients come from norm_rope_backward."""
    dev = _check_norm_rope(q, k, q_weight, k_weight, positions, freqs)
    p = make_norm_rope_problem(q, k, q_weight, freqs, eps, rot_offset, interleaved)
    c = _Call(stream, dev, q, k, q_weight, k_weight, positions, freqs)
    try:
        q_out = c.new(q.shape, q.dtype)
        k_out = None if k is None else c.new(k.shape, k.dtype)
        _check("csa_norm_rope", load().csa_norm_rope(
            ctypes.byref(p), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(positions), _ptr(freqs),
            _ptr(q_out), _ptr(k_out), c.handle))
    finally:
        c.done()
    return q_out, k_out


def norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, freqs, eps=1e-6, rot_offset=0,
                       interleaved=False, workspace=None, stream=None):
    """Gradients of norm_rope for the cotangents dq_out, dk_out (contiguous) ->
    (dq, dk, dq_weight, dk_weight): dq, dk contiguous in the inputs' type, the
    weights' gradients fp32 [D].  Without k: dk_out is None, and so are dk and
    dk_weight."""
    dev = _check_norm_rope(q, k, q_weight, k_weight, positions, freqs)
    _want(dq_out, "dq_out", q.shape, q.dtype, dev)
    if (dk_out is None) != (k is None):
        raise ValueError("dk_out and k come together")
    if k is not None:
        _want(dk_out, "dk_out", k.shape, q.dtype, dev)
    p = make_norm_rope_problem(q, k, q_weight, freqs, eps, rot_offset, interleaved)
    c = _Call(stream, dev, dq_out, dk_out, q, k, q_weight, k_weight, positions, freqs, workspace)
    try:
        D = q.shape[2]
        dq, dqw = c.new(q.shape, q.dtype), c.new((D,), torch.float32)
        dk = dkw = None
        if k is not None:
            dk, dkw = c.new(k.shape, k.dtype), c.new((D,), torch.float32)
        if workspace is None:
            workspace = c.new((int(load().csa_norm_rope_workspace_size(ctypes.byref(p))),), torch.uint8)
        _check("csa_norm_rope_backward", load().csa_norm_rope_backward(
            ctypes.byref(p), _ptr(dq_out), _ptr(dk_out), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
            _ptr(positions), _ptr(freqs), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw), _ptr(workspace),
            workspace.numel() * workspace.element_size(), c.handle))
    finally:
        c.done()
    return dq, dk, dqw, dkw


# ----------------------------------------------------------------------------- attention
def make_attn_problem(q, k, v, cu_q, scale, causal=True) -> AttnProblem:
    """Problem of q [Tq,Hq,D], k and v [Tk,Hk,D] and len(cu_q)-1 packed
    sequences; the tensors' strides are passed on."""
    Tq, Hq, D = q.shape
    p = AttnProblem(max(0, cu_q.numel() - 1), Tq, k.shape[0], Hq, k.shape[1], D, _dtype(q, "q"), 1 if causal else 0,
                    float(scale))
    p.q_stride_t, p.q_stride_h = _strides(q)
    p.k_stride_t, p.k_stride_h = _strides(k)
    p.v_stride_t, p.v_stride_h = _strides(v)
    return p


def attn_workspace_size(p: AttnProblem, which: int) -> int:
    return int(load().csa_attn_workspace_size(ctypes.byref(p), which))


def _check_attn(q, k, v, cu_q, cu_k, k_len):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [Tq, Hq, D], k and v [Tk, Hk, D]")
    dev = q.device
    _want(q, "q", q.shape, q.dtype, dev, True)
    _want(k, "k", (k.shape[0], k.shape[1], q.shape[2]), q.dtype, dev, True)
    _want(v, "v", k.shape, q.dtype, dev, True)
    n = cu_q.numel()
    if n < 1:
        raise ValueError("cu_q and cu_k hold one entry more than there are sequences")
    _want(cu_q, "cu_q", (n,), torch.int32, dev)
    _want(cu_k, "cu_k", (n,), torch.int32, dev)
    if k_len is not None:
        _want(k_len, "k_len", (n - 1,), torch.int32, dev)
    return dev


def attn_forward(q, k, v, cu_q, cu_k, scale, causal=True, k_len=None, workspace=None, stream=None):
    """Attention of packed sequences: q [Tq,Hq,D], k and v [Tk,Hk,D] (views
    allowed), cu_q and cu_k [N+1] int32 -> (out [Tq,Hq,D] in q's type,
    lse [Tq,Hq] fp32).  With k_len [N] int32 only the first k_len[i] keys of
    sequence i count: a cache [N,W,Hk,D] is passed as its view [N*W,Hk,D] with
    cu_k = arange(N+1)*W.  One query row per sequence is the decode step.  The
    outputs have no autograd history: gradients come from attn_backward."""
    dev = _check_attn(q, k, v, cu_q, cu_k, k_len)
    p = make_attn_problem(q, k, v, cu_q, scale, causal)
    c = _Call(stream, dev, q, k, v, cu_q, cu_k, k_len, workspace)
    try:
        out = c.new(q.shape, q.dtype)
        lse = c.new(q.shape[:2], torch.float32)
        if workspace is None:
            need = attn_workspace_size(p, 0)
            workspace = c.new((need,), torch.uint8) if need else None
        _check("csa_attn_forward", load().csa_attn_forward(
            ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(cu_q), _ptr(cu_k), _ptr(k_len), _ptr(out), _ptr(lse),
            _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), c.handle))
    finally:
        c.done()
    return out, lse


def attn_backward(dout, q, k, v, out, lse, cu_q, cu_k, scale, causal=True, k_len=None, workspace=None, stream=None):
    """Gradients of attn_forward for the cotangent dout of out (contiguous),
    from this forward's out and lse (not joined with other calls') -> (dq, dk, dv),
    contiguous, in q's type."""
    dev = _check_attn(q, k, v, cu_q, cu_k, k_len)
    _want(dout, "dout", q.shape, q.dtype, dev)
    _want(out, "out", q.shape, q.dtype, dev)
    _want(lse, "lse", q.shape[:2], torch.float32, dev)
    p = make_attn_problem(q, k, v, cu_q, scale, causal)
    c = _Call(stream, dev, dout, q, k, v, out, lse, cu_q, cu_k, k_len, workspace)
    try:
        dq = c.new(q.shape, q.dtype)
        dk, dv = c.new(k.shape, k.dtype), c.new(v.shape, v.dtype)
        if workspace is None:
            workspace = c.new((attn_workspace_size(p, 1),), torch.uint8)
        _check("csa_attn_backward", load().csa_attn_backward(
            ctypes.byref(p), _ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_q), _ptr(cu_k),
            _ptr(k_len), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
            workspace.numel() * workspace.element_size(), c.handle))
    finally:
        c.done()
    return dq, dk, dv
