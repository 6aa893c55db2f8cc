"""Norm and rotation of new tokens with their append to a paged cache, on the GPU.

q_out and the keys' rows are norm_rope's, bit for bit (the same arithmetic), and
norm_rope has its own test against the definition; one case is compared with the
definition here too, with that test's tolerance.  Values are copied: equal bits.
"""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu

BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    csa.load()


def _ok():
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK


def _bits(t):
    return t.view(torch.int32 if t.dtype == F32 else torch.int16)


def _case(new, past, page, Hq, Hk, D, dt, wt, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    T = sum(new)
    qkv = r(T, Hq + 2 * Hk, D).to(dt).cuda()
    k_len = [a + b for a, b in zip(new, past)]
    need = [-(-n // page) for n in k_len]
    order = np.random.default_rng(seed).permutation(sum(need) + 3)
    table = np.full((len(new), max(need, default=0) + 1), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    s = dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:], q_weight=(1 + 0.2 * r(D)).to(wt).cuda(),
             k_weight=(1 + 0.2 * r(D)).to(wt).cuda())
    s["positions"] = torch.tensor(np.concatenate([np.arange(a) + b for a, b in zip(new, past)] + [[]]).astype(np.int64)).cuda()
    s["cu_q"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    s["k_len"] = torch.tensor(k_len, dtype=torch.int32).cuda()
    s["k_pages"], s["v_pages"] = (r(len(order), page, Hk, D).to(dt).cuda() for _ in range(2))
    s["table"] = torch.tensor(table).cuda()
    rows = [table[i, j // page] * page + j % page for i, (a, b) in enumerate(zip(new, past)) for j in range(b, a + b)]
    return s, torch.tensor(rows, dtype=torch.int64).cuda()


def _call(s, freqs, **kw):
    return csa.norm_rope_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"], freqs, s["cu_q"],
                                s["k_len"], s["k_pages"], s["v_pages"], s["table"], **kw)


CASES = [  # new, past, page, Hq, Hk, D, rot, off, interleaved, dtype, wtype
    ([1], [0], 1, 1, 1, 8, 8, 0, True, BF, BF),
    ([1] * 9, [0, 1, 63, 64, 65, 127, 128, 5, 1000], 64, 64, 8, 128, 128, 0, False, BF, BF),
    ([0, 5, 0, 130, 1], [3, 60, 0, 7, 24], 24, 15, 5, 64, 32, 32, False, FP16, F32),
    ([70, 3], [0, 1], 7, 6, 2, 32, 16, 16, True, F32, F32),
    ([301], [11], 100, 3, 3, 256, 256, 0, False, BF, F32),
    ([4001, 0, 999], [0, 4, 2], 64, 2, 1, 128, 64, 0, True, BF, BF),
    ([33] * 40, [9] * 40, 16, 12, 3, 40, 32, 8, False, FP16, FP16),
    ([2500, 1700], [100, 0], 256, 9, 7, 128, 128, 0, False, F32, F32),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{sum(c[0])}x{c[3]}q{c[4]}k_D{c[5]}_{str(c[9])[6:]}_page{c[2]}")
def test_append(case):
    new, past, page, Hq, Hk, D, rot, off, inter, dt, wt = case
    s, rows = _case(new, past, page, Hq, Hk, D, dt, wt, seed=page)
    s["v"][0, 0, 0] = float("nan")
    s["v"][0, 0, 1:5] = torch.tensor([-0.0, float("inf"), -float("inf"), 1e-7], device="cuda").to(dt)
    fr = csa.rope_freqs(rot, 50000.0)
    arg = dict(eps=1e-5, rot_offset=off, interleaved=inter)
    yq, yk = csa.norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], fr, **arg)
    want_k, want_v = s["k_pages"].clone(), s["v_pages"].clone()
    want_k.view(-1, Hk, D)[rows], want_v.view(-1, Hk, D)[rows] = yk, s["v"]
    q_out = _call(s, fr, **arg)
    _ok()
    assert torch.equal(_bits(q_out), _bits(yq))
    assert torch.equal(_bits(s["k_pages"]), _bits(want_k)) and torch.equal(_bits(s["v_pages"]), _bits(want_v))


def test_against_the_definition():
    s, rows = _case([30, 1], [5, 77], 16, 4, 2, 64, BF, BF, seed=1)
    fr = csa.rope_freqs(64, 10000.0)
    q_out = _call(s, fr, eps=1e-6)
    _ok()
    ang = s["positions"].double().cpu().numpy()[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)[None]
    for x, w, got in ((s["q"], s["q_weight"], q_out), (s["k"], s["k_weight"], s["k_pages"].view(-1, 2, 64)[rows])):
        ref, mag = A.norm_rope(A.f64(x), A.f64(w), ang, 1e-6, 0, False)
        assert (np.abs(A.f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * mag + 1e-30).all()


def test_pools_side_by_side_and_strided_table():
    s, rows = _case([40, 3], [5, 77], 16, 4, 2, 64, BF, BF, seed=2)
    fr = csa.rope_freqs(64)
    both = torch.stack([s["k_pages"], s["v_pages"]], 1)
    wide = torch.cat([s["table"]] * 2, 1)
    t = dict(s, k_pages=both[:, 0], v_pages=both[:, 1], table=wide[:, :s["table"].shape[1]])
    a, b = _call(s, fr), _call(t, fr)
    _ok()
    assert torch.equal(a, b) and torch.equal(both[:, 0], s["k_pages"]) and torch.equal(both[:, 1], s["v_pages"])


def test_what_has_no_place_is_reported_and_not_stored():
    fr = csa.rope_freqs(64)
    for what in ("page", "negative_page", "short", "past_the_table"):
        s, rows = _case([6, 5], [20, 9], 8, 4, 2, 64, BF, BF, seed=3)
        full = dict(s, k_pages=s["k_pages"].clone(), v_pages=s["v_pages"].clone())
        want_q = _call(full, fr)
        _ok()
        t = dict(s, k_pages=s["k_pages"].clone(), v_pages=s["v_pages"].clone(), table=s["table"].clone(),
                 k_len=s["k_len"].clone())
        if what == "page":
            t["table"][1, 1] = t["k_pages"].shape[0]
        elif what == "negative_page":
            t["table"][1, 1] = -1
        elif what == "short":
            t["k_len"][1] = 3  # two of the five tokens stand before the sequence
        else:
            t["k_len"][1] = 8 * t["table"].shape[1] + 2
        got = _call(t, fr)
        torch.cuda.synchronize()
        assert csa.device_status() == csa.CSA_ERR_DEVICE, what
        assert torch.equal(got, want_q)
        if what in ("page", "negative_page"):
            want_k, want_v = s["k_pages"].clone(), s["v_pages"].clone()
            keep = torch.cat([torch.arange(6), torch.tensor([], dtype=torch.int64)])  # tokens 9..13 of sequence 1: page 1
            for w, x in ((want_k, full["k_pages"]), (want_v, full["v_pages"])):
                w.view(-1, 2, 64)[rows[keep]] = x.view(-1, 2, 64)[rows[keep]]
            assert torch.equal(t["k_pages"], want_k) and torch.equal(t["v_pages"], want_v)
        # rows of no new token are left as they were
        other = torch.ones(s["k_pages"].shape[0] * 8, dtype=torch.bool, device="cuda")
        other[rows] = False
        if what == "short":
            other[(s["table"][1, 0] * 8):(s["table"][1, 0] * 8 + 3)] = False
        if what != "past_the_table":
            assert torch.equal(t["k_pages"].view(-1, 2, 64)[other], s["k_pages"].view(-1, 2, 64)[other])


def test_tokens_of_no_sequence_are_turned_but_not_stored():
    s, rows = _case([6, 5], [20, 9], 8, 4, 2, 64, BF, BF, seed=4)
    fr = csa.rope_freqs(64)
    full = dict(s, k_pages=s["k_pages"].clone(), v_pages=s["v_pages"].clone())
    want = _call(full, fr)
    s["cu_q"][2] = 9  # the last two tokens belong to nobody
    s["k_len"][1] -= 2
    got = _call(s, fr)
    _ok()
    assert torch.equal(got, want)
    gone = rows[9:]
    assert not torch.equal(s["k_pages"], full["k_pages"])
    full["k_pages"].view(-1, 2, 64)[gone] = s["k_pages"].view(-1, 2, 64)[gone]
    assert torch.equal(s["k_pages"], full["k_pages"])


def test_replayed_from_a_graph_and_another_stream():
    s, rows = _case([1] * 5, [20, 9, 3, 0, 1], 8, 4, 2, 64, BF, BF, seed=5)
    fr = csa.rope_freqs(64)
    want = dict(s, k_pages=s["k_pages"].clone(), v_pages=s["v_pages"].clone())
    want_q = _call(want, fr)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    one = dict(s, k_pages=s["k_pages"].clone(), v_pages=s["v_pages"].clone())
    torch.cuda.synchronize()
    got_q = _call(one, fr, stream=side)
    side.synchronize()
    assert torch.equal(got_q, want_q) and torch.equal(one["k_pages"], want["k_pages"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _call(s, fr)
    for _ in range(2):
        g.replay()
    _ok()
    assert torch.equal(out, want_q) and torch.equal(s["k_pages"], want["k_pages"]) and torch.equal(s["v_pages"], want["v_pages"])
