"""Host-side checks of include/csa_sparse.h (no GPU, no compute calls): every
declared entry point is exported, and bad arguments are refused before any
CUDA call."""
import ctypes
import os
import re

import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from sparse_attention_indexer_csa_gb300 import abi, attn, sparse

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)  # 16-byte aligned, never dereferenced by the checks
ODD = ctypes.c_void_p(0x10002)
BYTE = ctypes.c_void_p(0x10001)
OK, INVALID, UNSUPPORTED = abi.CSA_OK, abi.CSA_ERR_INVALID_ARG, abi.CSA_ERR_UNSUPPORTED
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from sparse_attention_indexer_csa_gb300 import build
        build.build()
    return sparse.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "csa_sparse.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(csa_[a-z_]+)\s*\(", text))
    assert names == set(sparse.EXPORTED)
    for n in names:
        assert hasattr(lib, n), n
    assert lib.csa_sparse_abi_version() == 100


# ----------------------------------------------------------------------------- attention over listed blocks
def _sp(**kw):
    d = dict(N=2, Tq=10, Tk=20, Hq=8, Hk=2, D=128, top_k=3, block=4, window=5, page=0, table_width=0,
             dtype=abi.CSA_BF16, causal=1, scale=0.1)
    d.update(kw)
    return sparse.SparseProblem(**d)


def _paged(**kw):
    return _sp(**{**dict(page=5, table_width=4), **kw})


def _fwd(lib, p, ws_bytes=BIG, **kw):
    names = ("q", "k", "v", "idx", "cq", "ck", "kl", "table", "out", "lse", "ws")
    paged = p is not None and p.page > 0
    none = ("ck",) if paged else ("kl", "table")
    a = {x: kw.get(x, None if x in none else FAKE) for x in names}
    return lib.csa_sparse_attn_forward(ctypes.byref(p) if p is not None else None, *[a[x] for x in names], ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(N=-1), dict(Tq=-1), dict(Tk=-1), dict(Hq=0), dict(Hk=0), dict(D=0), dict(Hk=3),
                                 dict(top_k=-1), dict(block=0), dict(block=-4), dict(window=-1), dict(page=-1),
                                 dict(table_width=-1), dict(table_width=2), dict(dtype=9), dict(causal=2),
                                 dict(causal=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
                                 dict(idx_stride=2), dict(idx_stride=-3), dict(table_stride=-1), dict(q_stride_t=4),
                                 dict(q_stride_h=-8), dict(k_stride_t=1 << 40), dict(k_stride_h=12), dict(v_stride_t=-128),
                                 dict(v_stride_h=2), dict(k_stride_p=4), dict(v_stride_p=-8),
                                 dict(page=6, table_width=4), dict(page=5, table_width=4, table_stride=3)])
def test_sparse_bad_problem(lib, bad):
    assert _fwd(lib, _sp(**bad)) == INVALID
    for which in (0, 1):
        assert lib.csa_sparse_attn_workspace_size(ctypes.byref(_sp(**bad)), which) == 0


@pytest.mark.parametrize("bad", [dict(D=96), dict(D=32), dict(D=256), dict(dtype=abi.CSA_F32), dict(Hq=258, Hk=2),
                                 dict(block=3), dict(block=256), dict(window=1 << 20), dict(top_k=1 << 19),
                                 dict(Tk=2_000_000_000, Hk=8), dict(k_stride_t=8 * 1000_000_007, k_stride_h=8)])
def test_sparse_unsupported(lib, bad):
    assert _fwd(lib, _sp(**bad)) == UNSUPPORTED
    for which in (0, 1):
        assert lib.csa_sparse_attn_workspace_size(ctypes.byref(_sp(**bad)), which) == 0


def test_sparse_pointers(lib):
    assert _fwd(lib, None) == INVALID
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(idx=None), dict(cq=None), dict(ck=None), dict(out=None),
               dict(lse=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(idx=BYTE), dict(cq=BYTE), dict(ck=BYTE),
               dict(kl=ODD), dict(out=ODD), dict(lse=ctypes.c_void_p(0x10008)), dict(table=FAKE)):
        assert _fwd(lib, _sp(), **kw) == INVALID, kw
    assert _fwd(lib, _sp(top_k=0)) == INVALID  # a list without places
    # paged: no cu_k, and lengths and the table
    for kw in (dict(ck=FAKE), dict(kl=None), dict(table=None), dict(table=BYTE)):
        assert _fwd(lib, _paged(), **kw) == INVALID, kw
    # few rows and a long list need a workspace
    long = _sp(Tq=1, N=1, Tk=100000, top_k=1000)
    need = int(lib.csa_sparse_attn_workspace_size(ctypes.byref(long), 0))
    assert need > 0
    assert _fwd(lib, long, ws=None) == INVALID and _fwd(lib, long, need - 1) == INVALID
    assert _fwd(lib, long, ws=ctypes.c_void_p(0x10008)) == INVALID
    # no query row: nothing is enqueued
    assert _fwd(lib, _sp(Tq=0), q=None, out=None, lse=None, idx=None) == OK


def _bwd(lib, p, ws_bytes=BIG, **kw):
    names = ("do", "q", "k", "v", "out", "lse", "idx", "cq", "ck", "kl", "dq", "dk", "dv", "ws")
    a = {x: kw.get(x, None if x == "kl" else FAKE) for x in names}
    return lib.csa_sparse_attn_backward(ctypes.byref(p), *[a[x] for x in names], ws_bytes, None)


def test_sparse_backward_refusals(lib):
    for x in ("do", "q", "k", "v", "out", "lse", "idx", "cq", "ck", "dq", "dk", "dv", "ws"):
        assert _bwd(lib, _sp(), **{x: None}) == INVALID, x
    for x in ("do", "out", "dq", "dk", "dv"):
        assert _bwd(lib, _sp(), **{x: ODD}) == INVALID, x
    need = int(lib.csa_sparse_attn_workspace_size(ctypes.byref(_sp()), 1))
    assert need > 0 and _bwd(lib, _sp(), need - 1) == INVALID
    assert _bwd(lib, _sp(D=32)) == UNSUPPORTED
    assert _bwd(lib, _paged()) == UNSUPPORTED  # the cache takes no gradients
    empty = _sp(Tq=0, Tk=0)
    assert _bwd(lib, empty, do=None, q=None, k=None, v=None, out=None, lse=None, idx=None, dq=None, dk=None, dv=None) == OK


def test_sparse_workspace_stays_within_its_limit(lib):
    # a long list: rounds of as many rows as 4 GiB hold, and sums, counts and entries beside them
    p = _sp(N=1, Tq=65536, Tk=65536, Hq=64, Hk=8, top_k=1024, block=1, window=0)
    need = int(lib.csa_sparse_attn_workspace_size(ctypes.byref(p), 1))
    assert 2 << 30 < need < (4 << 30) + 8 * 65536 * 8 * 128 + 3 * 65536 * 64 * 4 + (1 << 30)


# ----------------------------------------------------------------------------- append to a paged cache
def _np(**kw):
    d = dict(T=5, Hq=4, Hk=2, D=64, rot=64, rot_offset=0, interleaved=0, dtype=abi.CSA_BF16, w_dtype=abi.CSA_BF16,
             eps=1e-6)
    d.update(kw)
    return attn.NormRopeProblem(**d)


def _cp(**kw):
    d = dict(N=2, pages=7, page=16, table_width=3)
    d.update(kw)
    return sparse.AppendProblem(**d)


def _app(lib, p, c, **kw):
    names = ("q", "k", "v", "qw", "kw", "pos", "fr", "cq", "kl", "table", "yq", "kc", "vc")
    return lib.csa_norm_rope_append(ctypes.byref(p) if p is not None else None, ctypes.byref(c) if c is not None else None,
                                    *[kw.get(x, FAKE) for x in names], None)


def test_append_refusals(lib):
    assert _app(lib, None, _cp()) == INVALID and _app(lib, _np(), None) == INVALID
    for bad in (dict(T=-1), dict(Hk=0), dict(rot=7), dict(dtype=3), dict(eps=-1.0), dict(q_stride_t=12)):
        assert _app(lib, _np(**bad), _cp()) == INVALID, bad
    assert _app(lib, _np(rot=24), _cp()) == UNSUPPORTED
    for bad in (dict(N=-1), dict(pages=-1), dict(page=0), dict(table_width=-1), dict(table_stride=2),
                dict(table_stride=-3), dict(v_stride_t=4), dict(v_stride_h=-8), dict(kc_stride_p=4), dict(kc_stride_t=12),
                dict(vc_stride_h=1 << 40)):
        assert _app(lib, _np(), _cp(**bad)) == INVALID, bad
    for x in ("q", "k", "v", "qw", "kw", "pos", "fr", "cq", "kl", "table", "yq", "kc", "vc"):
        assert _app(lib, _np(), _cp(), **{x: None}) == INVALID, x
    for x in ("q", "k", "v", "pos", "fr", "cq", "kl", "table", "yq", "kc", "vc"):
        assert _app(lib, _np(), _cp(), **{x: BYTE}) == INVALID, x
    # no token: nothing is enqueued
    none = dict.fromkeys(("q", "k", "v", "pos", "yq", "kc", "vc"))
    assert _app(lib, _np(T=0), _cp(), **none) == OK


# ----------------------------------------------------------------------------- binding
def test_binding_refuses_host_tensors_and_wrong_shapes():
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    idx, cu = torch.zeros(3, 2, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        csa.sparse_attn_forward(q, q, q, idx, cu, cu, 0.1)
    with pytest.raises(ValueError):
        csa.sparse_attn_forward(q[0], q, q, idx, cu, cu, 0.1)
    with pytest.raises(ValueError, match="GPU"):
        csa.sparse_attn_backward(q, q, q, q, q, q[..., 0].float(), idx, cu, cu, 0.1)
    with pytest.raises(ValueError, match="GPU"):
        csa.sparse_attn_paged(q, q[None], q[None], idx[:1], idx, cu, cu[1:], 0.1)
    w, pos, fr = torch.ones(64), torch.zeros(3, dtype=torch.int64), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError):
        csa.norm_rope_append(q, None, None, w, None, pos, fr, cu, cu[1:], q[None], q[None], idx[:1])
    with pytest.raises(ValueError, match="GPU"):
        csa.norm_rope_append(q, q, q, w, w, pos, fr, cu, cu[1:], q[None], q[None], idx[:1])


def test_problem_of_views_carries_their_strides():
    qkv = torch.zeros(7, 10, 64, dtype=torch.float16)
    idx, cu = torch.zeros(7, 9, dtype=torch.int32)[:, 2:5], torch.tensor([0, 7], dtype=torch.int32)
    p = csa.make_sparse_problem(qkv[:, :6], qkv[:, 6:8], qkv[:, 8:], idx, cu, 0.5, block=2, window=3)
    assert (p.N, p.Tq, p.Tk, p.Hq, p.Hk, p.D, p.top_k, p.block, p.window, p.page) == (1, 7, 7, 6, 2, 64, 3, 2, 3, 0)
    assert (p.dtype, p.causal, p.scale, p.idx_stride) == (attn.CSA_F16, 1, 0.5, 9)
    assert (p.q_stride_t, p.q_stride_h, p.k_stride_t, p.k_stride_h, p.v_stride_t, p.v_stride_h) == (640, 64) * 3
    pool = torch.zeros(5, 2, 8, 3, 64, dtype=torch.float16)
    table = torch.zeros(1, 6, dtype=torch.int32)[:, :4]
    p = csa.make_sparse_problem(qkv[:, :6], pool[:, 0], pool[:, 1], None, cu, 0.5, causal=False, table=table)
    assert (p.Tk, p.Hk, p.page, p.table_width, p.top_k, p.causal) == (40, 3, 8, 4, 0, 0)
    assert (p.k_stride_p, p.k_stride_t, p.k_stride_h) == (2 * 8 * 3 * 64, 192, 64)
