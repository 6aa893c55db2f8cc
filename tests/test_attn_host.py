"""Host-side checks of include/csa_attn.h (no GPU, no compute calls): every
declared entry point is exported, and bad arguments are refused before any
CUDA call."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from sparse_attention_indexer_csa_gb300 import abi, attn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)  # 16-byte aligned, never dereferenced by the checks
ODD = ctypes.c_void_p(0x10002)
OK, INVALID, UNSUPPORTED = abi.CSA_OK, abi.CSA_ERR_INVALID_ARG, abi.CSA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from sparse_attention_indexer_csa_gb300 import build
        build.build()
    return attn.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "csa_attn.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(csa_[a-z_]+)\s*\(", text))
    assert names == set(attn.EXPORTED)
    for n in names:
        assert hasattr(lib, n), n
    assert lib.csa_attn_abi_version() == 100


# ----------------------------------------------------------------------------- frequencies
def test_rope_freqs_are_the_fractions_of_a_turn(lib):
    t = csa.rope_freqs(64, 10000.0, device="cpu").numpy().view(np.uint64)
    for i, f in enumerate(t):
        want = 10000.0 ** (-2 * i / 64) / (2 * math.pi)
        # a few roundings of 64-bit floating point, and the table's own step of 2^-64
        assert abs(float(f) / 2.0 ** 64 - want) <= want * 2 ** -51 + 2.0 ** -64


@pytest.mark.parametrize("theta,rot", [(1.0, 64), (0.5, 64), (float("nan"), 64), (float("inf"), 64), (1e4, 63), (1e4, 0)])
def test_rope_freqs_refusals(lib, theta, rot):
    with pytest.raises(csa.CsaError):
        csa.rope_freqs(rot, theta, device="cpu")


# ----------------------------------------------------------------------------- norm + rotation
def _np(**kw):
    d = dict(T=5, Hq=4, Hk=2, D=64, rot=64, rot_offset=0, interleaved=0, dtype=abi.CSA_BF16, w_dtype=abi.CSA_BF16,
             eps=1e-6)
    d.update(kw)
    return attn.NormRopeProblem(**d)


def _nr(lib, p, q=FAKE, k=FAKE, qw=FAKE, kw=FAKE, pos=FAKE, fr=FAKE, yq=FAKE, yk=FAKE):
    return lib.csa_norm_rope(ctypes.byref(p) if p is not None else None, q, k, qw, kw, pos, fr, yq, yk, None)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(D=0), dict(rot=0), dict(rot=7),
                                 dict(rot_offset=-8), dict(rot_offset=8), dict(rot=128), dict(interleaved=2),
                                 dict(dtype=3), dict(w_dtype=-1), dict(eps=-1.0), dict(eps=float("nan")),
                                 dict(eps=float("inf")), dict(q_stride_t=-8), dict(q_stride_h=4), dict(k_stride_t=12),
                                 dict(k_stride_h=1 << 40), dict(dtype=abi.CSA_F32, q_stride_t=2)])
def test_norm_rope_bad_problem(lib, bad):
    assert _nr(lib, _np(**bad)) == INVALID


@pytest.mark.parametrize("bad", [dict(D=60, rot=16), dict(D=264, rot=16), dict(rot=16, rot_offset=4), dict(rot=24),
                                 dict(rot=12, interleaved=1)])
def test_norm_rope_unsupported(lib, bad):
    assert _nr(lib, _np(**bad)) == UNSUPPORTED


def test_norm_rope_pointers(lib):
    assert _nr(lib, None) == INVALID
    for kw in (dict(q=None), dict(k=None), dict(qw=None), dict(kw=None), dict(pos=None), dict(fr=None), dict(yq=None),
               dict(yk=None), dict(q=ODD), dict(k=ODD), dict(yq=ODD), dict(yk=ODD), dict(pos=ODD), dict(fr=ODD)):
        assert _nr(lib, _np(), **kw) == INVALID, kw
    # without keys their pointers have to be NULL
    assert _nr(lib, _np(Hk=0)) == INVALID
    # no token: nothing is enqueued
    assert _nr(lib, _np(T=0), q=None, k=None, pos=None, yq=None, yk=None) == OK


def _nb(lib, p, nbytes=None, **kw):
    names = ("gq", "gk", "q", "k", "qw", "kw", "pos", "fr", "dq", "dk", "dqw", "dkw", "ws")
    a = {n: kw.get(n, FAKE) for n in names}
    nbytes = int(lib.csa_norm_rope_workspace_size(ctypes.byref(p))) if nbytes is None else nbytes
    return lib.csa_norm_rope_backward(ctypes.byref(p), *[a[n] for n in names], nbytes, None)


def test_norm_rope_backward_refusals(lib):
    assert lib.csa_norm_rope_workspace_size(ctypes.byref(_np())) == 152 * 4 * 2 * 64 * 4
    assert lib.csa_norm_rope_workspace_size(ctypes.byref(_np(D=0))) == 0
    for n in ("gq", "gk", "q", "k", "qw", "kw", "pos", "fr", "dq", "dk", "dqw", "dkw", "ws"):
        assert _nb(lib, _np(), **{n: None}) == INVALID, n
    assert _nb(lib, _np(), ws=ctypes.c_void_p(0x10008)) == INVALID
    assert _nb(lib, _np(), nbytes=16) == INVALID
    assert _nb(lib, _np(rot=24)) == UNSUPPORTED


# ----------------------------------------------------------------------------- attention
def _ap(**kw):
    d = dict(N=2, Tq=10, Tk=20, Hq=8, Hk=2, D=128, dtype=abi.CSA_BF16, causal=1, scale=0.1)
    d.update(kw)
    return attn.AttnProblem(**d)


WS = 1 << 40


def _af(lib, p, q=FAKE, k=FAKE, v=FAKE, cq=FAKE, ck=FAKE, kl=None, out=FAKE, lse=FAKE, ws=FAKE, n=WS):
    return lib.csa_attn_forward(ctypes.byref(p) if p is not None else None, q, k, v, cq, ck, kl, out, lse, ws, n, None)


@pytest.mark.parametrize("bad", [dict(N=-1), dict(Tq=-1), dict(Tk=-1), dict(Hq=0), dict(Hk=0), dict(D=0), dict(Hk=3),
                                 dict(dtype=9), dict(causal=2), dict(scale=0.0), dict(scale=-1.0),
                                 dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride_t=4),
                                 dict(q_stride_h=-8), dict(k_stride_t=1 << 40), dict(k_stride_h=12),
                                 dict(v_stride_t=-128), dict(v_stride_h=2)])
def test_attn_bad_problem(lib, bad):
    assert _af(lib, _ap(**bad)) == INVALID
    assert lib.csa_attn_workspace_size(ctypes.byref(_ap(**bad)), 1) == 0


@pytest.mark.parametrize("bad", [dict(D=96), dict(D=32), dict(D=256), dict(dtype=abi.CSA_F32),
                                 dict(Hq=258, Hk=2), dict(Tk=2_000_000_000, Hk=8)])
def test_attn_unsupported(lib, bad):
    assert _af(lib, _ap(**bad)) == UNSUPPORTED


def test_attn_pointers(lib):
    assert _af(lib, None) == INVALID
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(cq=None), dict(ck=None), dict(out=None), dict(lse=None),
               dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(cq=ctypes.c_void_p(0x10001)), dict(kl=ODD), dict(out=ODD),
               dict(lse=ctypes.c_void_p(0x10008))):
        assert _af(lib, _ap(), **kw) == INVALID, kw
    # no query row: nothing is enqueued
    assert _af(lib, _ap(Tq=0), q=None, out=None, lse=None) == OK


def _ab(lib, p, n=WS, **kw):
    names = ("do", "q", "k", "v", "out", "lse", "cq", "ck", "kl", "dq", "dk", "dv", "ws")
    a = {x: kw.get(x, None if x == "kl" else FAKE) for x in names}
    return lib.csa_attn_backward(ctypes.byref(p), *[a[x] for x in names], n, None)


def test_attn_backward_refusals(lib):
    for x in ("do", "q", "k", "v", "out", "lse", "cq", "ck", "dq", "dk", "dv", "ws"):
        assert _ab(lib, _ap(), **{x: None}) == INVALID, x
    for x in ("do", "out", "dq", "dk", "dv"):
        assert _ab(lib, _ap(), **{x: ODD}) == INVALID, x
    need = int(lib.csa_attn_workspace_size(ctypes.byref(_ap()), 1))
    assert need > 0 and _ab(lib, _ap(), n=need - 1) == INVALID
    assert _ab(lib, _ap(D=32)) == UNSUPPORTED
    empty = _ap(Tq=0, Tk=0)
    assert _ab(lib, empty, do=None, q=None, k=None, v=None, out=None, lse=None, dq=None, dk=None, dv=None) == OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        csa.attn_forward(q, q, q, cu, cu, 0.1)
    with pytest.raises(ValueError):
        csa.norm_rope(q, None, torch.ones(64), torch.ones(64), torch.zeros(3, dtype=torch.int64),
                      torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError):
        csa.attn_forward(q[0], q, q, cu, cu, 0.1)
