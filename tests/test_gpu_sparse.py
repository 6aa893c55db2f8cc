"""Attention over listed blocks of keys on the GPU against the fp64 definition: packed, paged, forward and gradients.

Tolerances, from the arithmetic (u = eps/2 of the storage type), as for dense attention:
* scores: an error ds of at most 2^-16 of the row's largest scale*|q|.|k| (fp32 sums of up to 128 products).
* p is off by 2 ds relative, 2^-20 for the exponential, and u where it is rounded for the product with v; the sum (fp32)
  by the same but u; the join of shares adds a few fp32 roundings: 2^-18 in all.
      |out - ref| <= u |ref| + (u + 2 ds + 2^-18) sum p|v| + tiny sum |v|
      |lse - ref| <= ds + 2^-19 + 2^-22 |ref|
* gradients: as above with ds rounded to the storage type and delta from the rounded out (u each), and, in bf16, the shares
  of the rows in dk and dv rounded to fp16 at a power of two that their bound (norm_dk, norm_dv) is at most twice below: 2^-11 of
  their magnitude, 2^-25 of 2^-15 of twice the bound where fp16 has no more bits:
      |dq - ref| <= u |ref| + (2u + 2 ds + 2^-15) mag + tiny (sum of the other factor)
      dk: 2u + 2^-11 + ... and 2^-39 norm_dk;  dv: u + 2^-11 + 2 ds + 2^-18 and 2^-39 norm_dv  (fp16: without these).
* fp16 weights are formed at 2^8 (in out) and 2^15 (in dv) of their size, and ds at a power of two that brings its
  bound above 2^13: subnormal spacing 2^-24, so tiny is 2^-33 per key in out, 2^-40 in dv, 2^-38 of ds' bound in
  dq and dk.  bf16 has fp32's range: 0.
* rounding a result x to fp16 is off by u |x| for |x| >= 2^-14 and, below, where fp16's numbers are 2^-24 apart, by half
  of that: 2^-25 is added to every fp16 bound.  (bf16's subnormals start at 2^-126: the 1e-30 of _check.)
"""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from oracle import sparse_oracle as S
from oracle.attn_oracle import f64

pytestmark = pytest.mark.gpu

BF, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    csa.load()


def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)


def _inputs(lq, lk, Hq, Hk, D, dt, seed=0, size=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=gen) * size).to(dt)  # noqa: E731
    return r(sum(lq), Hq, D), r(sum(lk), Hk, D), r(sum(lk), Hk, D), r(sum(lq), Hq, D)


def _lists(lq, lk, K, block, seed=0, holes=0.2):
    """Distinct blocks of each row's sequence in any order, some places empty."""
    rng = np.random.default_rng(seed)
    idx = np.full((sum(lq), K), -1, dtype=np.int32)
    t = 0
    for a, b in zip(lq, lk):
        nb = -(-b // block)
        for _ in range(a):
            n = min(K, nb)
            some = rng.permutation(nb)[:n]
            at = rng.permutation(K)[:n]
            idx[t, at] = np.where(rng.random(n) < holes, -1, some)
            t += 1
    return torch.tensor(idx)


def _check(name, got, want, bound):
    g = f64(got)
    assert np.array_equal(np.isneginf(g), np.isneginf(want)), name
    fin = ~np.isneginf(want)
    assert np.isfinite(g[fin]).all(), name
    err = np.abs(np.where(fin, g, 0) - np.where(fin, want, 0))
    r = err / (np.where(fin, bound, 1) + 1e-30)
    assert r.max(initial=0.0) <= 1.0, (name, float(r.max()), np.unravel_index(r.argmax(), r.shape))


def _bounds(ref, dt):
    u = torch.finfo(dt).eps / 2
    h = 1.0 if dt == FP16 else 0.0
    ds = 2.0 ** -16 * ref["smax"]
    lse = np.where(np.isneginf(ref["lse"]), 0, ref["lse"])
    b = dict(out=u * np.abs(ref["out"]) + (u + 2 * ds[..., None] + 2.0 ** -18) * ref["mag_out"]
             + h * (2.0 ** -33 * ref["vsum"] + 2.0 ** -25), lse=ds + 2.0 ** -19 + 2.0 ** -22 * np.abs(lse))
    top = 2 * ds.max(initial=0.0)
    sh = 0.0 if dt == FP16 else 1.0
    rel = dict(dq=2 * u + top + 2.0 ** -15, dk=2 * u + sh * 2.0 ** -11 + top + 2.0 ** -15,
               dv=u + sh * 2.0 ** -11 + top + 2.0 ** -18)
    tiny = dict(dq=2.0 ** -38, dk=2.0 ** -38, dv=2.0 ** -40)
    for n in ("dq", "dk", "dv"):
        if n in ref:
            share = sh * 2.0 ** -39 * ref["norm_" + n][..., None] if n != "dq" else 0.0
            b[n] = u * np.abs(ref[n]) + rel[n] * ref["mag_" + n] + share + h * (tiny[n] * ref["sum_" + n] + 2.0 ** -25)
    return b


def _ok():
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK


def _run(q, k, v, do, idx, cu_q, cu_k, scale, backward=True, k_len=None, **kw):
    """Forward and gradients on the GPU, checked against the definition."""
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    a = [c(t) for t in (idx, cu_q, cu_k)]
    out, lse = csa.sparse_attn_forward(c(q), c(k), c(v), *a, scale, k_len=c(k_len), **kw)
    _ok()
    n = lambda t: None if t is None else t.numpy()  # noqa: E731
    lists = np.zeros((q.shape[0], 0), dtype=np.int32) if idx is None else n(idx)
    ref = S.attention(f64(q), f64(k), f64(v), lists, n(cu_q), n(cu_k), scale, k_len=n(k_len),
                      dout=f64(do) if backward else None, **kw)
    b = _bounds(ref, q.dtype)
    _check("out", out, ref["out"], b["out"])
    _check("lse", lse, ref["lse"], b["lse"])
    if not backward:
        return out, lse
    grads = csa.sparse_attn_backward(c(do), c(q), c(k), c(v), out, lse, *a, scale, k_len=c(k_len), **kw)
    _ok()
    for name, t in zip(("dq", "dk", "dv"), grads):
        _check(name, t, ref[name], b[name])
    return out, lse, *grads


LENGTHS = {
    "one": ([1], [1]),
    "tile_edges": ([1, 2, 3], [127, 128, 129]),
    "empty_ones": ([0, 5, 0, 0, 70, 0], [0, 5, 9, 0, 70, 0]),
    "no_keys": ([4, 3], [0, 3]),
    "rows_without_keys": ([100, 40], [60, 39]),
    "behind_a_prefix": ([1, 33, 7], [300, 500, 129]),
}
# heads, K, block, window
SHAPES = [(1, 1, 128, BF, 1, 1, 0), (8, 1, 64, FP16, 33, 2, 5), (6, 2, 128, FP16, 130, 1, 0), (12, 4, 64, BF, 5, 64, 1),
          (64, 2, 128, BF, 17, 16, 40), (64, 1, 128, BF, 200, 1, 0), (100, 1, 64, FP16, 9, 8, 130),
          (128, 1, 128, BF, 70, 4, 0), (66, 2, 64, BF, 3, 128, 0), (7, 7, 128, BF, 40, 4, 128)]


def _shape_id(s):
    return f"{s[0]}q{s[1]}k_D{s[2]}_{str(s[3])[6:]}_K{s[4]}x{s[5]}_w{s[6]}"


@pytest.mark.parametrize("shape", SHAPES, ids=_shape_id)
@pytest.mark.parametrize("lengths", LENGTHS)
def test_forward(lengths, shape):
    lq, lk = LENGTHS[lengths]
    Hq, Hk, D, dt, K, block, window = shape
    q, k, v, do = _inputs(lq, lk, Hq, Hk, D, dt, seed=len(lq) + D)
    idx = _lists(lq, lk, K, block, seed=K)
    _run(q, k, v, do, idx, _cu(lq), _cu(lk), D ** -0.5, backward=False, block=block, window=window)


@pytest.mark.parametrize("shape", SHAPES[:8], ids=_shape_id)
def test_forward_without_causal_border(shape):
    Hq, Hk, D, dt, K, block, _ = shape
    lq, lk = [5, 40, 0, 3, 1], [70, 129, 3, 257, 0]
    q, k, v, do = _inputs(lq, lk, Hq, Hk, D, dt, seed=3)
    idx = _lists(lq, lk, K, block, seed=5)
    _run(q, k, v, do, idx, _cu(lq), _cu(lk), D ** -0.5, backward=False, block=block, causal=False)


def test_window_alone_is_sliding_attention():
    lq = [70, 1, 300]
    q, k, v, do = _inputs(lq, lq, 4, 2, 64, BF, seed=9)
    one = _run(q, k, v, do, None, _cu(lq), _cu(lq), 0.125, backward=False, window=50)
    none = torch.full((sum(lq), 3), -1, dtype=torch.int32)
    two = _run(q, k, v, do, none, _cu(lq), _cu(lq), 0.125, backward=False, window=50)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_large_scores_and_the_reference():
    # scores up to several hundred, growing and falling along the list: tiles raise the reference
    q, k, v, do = _inputs([9], [900], 4, 1, 128, BF, seed=8, size=2.0)
    idx = torch.arange(900, dtype=torch.int32).repeat(9, 1)
    for steep in (torch.linspace(0.1, 4.0, 900), torch.linspace(4.0, 0.1, 900)):
        kk = (k.float() * steep[:, None, None]).to(BF)
        _run(q, kk, v, do, idx, _cu([9]), _cu([900]), 1.0, backward=False, causal=False)


@pytest.mark.parametrize("N,W,K,Hq,Hk,D,dt", [(1, 9000, 3000, 8, 1, 128, BF), (3, 5000, 1023, 6, 2, 64, FP16),
                                              (2, 20001, 2000, 64, 1, 128, BF), (5, 3000, 700, 128, 1, 64, FP16)])
def test_few_rows_with_long_lists(N, W, K, Hq, Hk, D, dt):
    lq, lk = [1] * N, [W] * N
    q, k, v, do = _inputs(lq, lk, Hq, Hk, D, dt, seed=W)
    idx = _lists(lq, lk, K, 1, seed=W)
    _run(q, k, v, do, idx, _cu(lq), _cu(lk), D ** -0.5, backward=False)


def test_a_block_listed_twice_counts_twice():
    q, k, v, do = _inputs([3], [40], 4, 2, 64, BF, seed=4)
    idx = torch.tensor([[3, 3, 1, -1], [0, 2, 0, 0], [5, 5, 5, 5]], dtype=torch.int32)
    _run(q, k, v, do, idx, _cu([3]), _cu([40]), 0.2, backward=False, block=4, causal=False)


def test_hidden_keys_may_hold_anything():
    lq, lk = [6, 30], [200, 100]
    q, k, v, _ = _inputs(lq, lk, 8, 2, 128, BF, seed=6)
    k_len = torch.tensor([150, 100], dtype=torch.int32)
    idx = _lists(lq, [150, 100], 20, 2, seed=1)
    c = lambda t: t.cuda()  # noqa: E731
    call = lambda: csa.sparse_attn_forward(c(q), c(k), c(v), c(idx), c(_cu(lq)), c(_cu(lk)), 0.1, block=2, window=9,  # noqa: E731
                                           k_len=c(k_len))
    want = call()
    seen = np.zeros(sum(lk), dtype=bool)
    n = [S.counts(idx.numpy()[:6], np.arange(6) + 144, 150, 2, 9, True),
         S.counts(idx.numpy()[6:], np.arange(30) + 70, 100, 2, 9, True)]
    seen[:150], seen[200:] = n[0].any(0), n[1].any(0)
    hidden = torch.tensor(~seen)
    assert hidden.sum() > 50
    for bad in (float("nan"), float("inf"), -float("inf")):
        k[hidden], v[hidden] = bad, bad
        got = call()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    # a key that one row sees and the other rows do not: only that row changes
    v[0] = float("nan")
    got = call()
    rows = torch.tensor(np.concatenate([n[0][:, 0] > 0, np.zeros(30, dtype=bool)])).cuda()
    assert torch.equal(got[0][~rows], want[0][~rows]) and (rows.sum() == 0 or got[0][rows].isnan().any())
    _ok()


def test_views_and_strided_lists():
    T, Hq, Hk, D, K = 77, 6, 3, 64, 11
    gen = torch.Generator().manual_seed(12)
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=gen).to(FP16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    wide = torch.full((T, K + 6), 10 ** 6, dtype=torch.int32)
    idx = _lists([T], [T], K, 2, seed=2)
    wide[:, 3:3 + K] = idx
    g = qkv.cuda()
    args = (_cu([T]).cuda(), _cu([T]).cuda(), 0.125)
    got = csa.sparse_attn_forward(g[:, :Hq], g[:, Hq:Hq + Hk], g[:, Hq + Hk:], wide.cuda()[:, 3:3 + K], *args, block=2)
    want = csa.sparse_attn_forward(*(t.contiguous().cuda() for t in (q, k, v)), idx.cuda(), *args, block=2)
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # heads in front of tokens
    kt, vt = (t.contiguous().cuda().transpose(0, 1).contiguous().transpose(0, 1) for t in (k, v))
    got = csa.sparse_attn_forward(q.contiguous().cuda(), kt, vt, idx.cuda(), *args, block=2)
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bad_lists_are_reported_and_skipped():
    lq, lk = [4, 5], [30, 20]
    q, k, v, _ = _inputs(lq, lk, 4, 1, 64, BF, seed=13)
    idx = _lists(lq, lk, 6, 4, seed=3, holes=0.0)
    bad = idx.clone()
    bad[:, 2] = -1
    args = (_cu(lq).cuda(), _cu(lk).cuda(), 0.125)
    call = lambda i: csa.sparse_attn_forward(q.cuda(), k.cuda(), v.cuda(), i.cuda(), *args, block=4, causal=False)  # noqa: E731
    want = call(bad)
    _ok()
    for value in (-2, 8, 2 ** 31 - 1, -2 ** 31):
        bad[:, 2] = value
        got = call(bad)
        torch.cuda.synchronize()
        assert csa.device_status() == csa.CSA_ERR_DEVICE
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    _ok()


def test_rows_outside_every_sequence_and_bad_borders():
    q, k, v, _ = _inputs([10], [10], 2, 1, 64, BF, seed=14)
    idx = torch.zeros(10, 1, dtype=torch.int32)
    c = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    call = lambda a, b: csa.sparse_attn_forward(q.cuda(), k.cuda(), v.cuda(), idx.cuda(), a, b, 0.125)  # noqa: E731
    out, lse = call(c([2, 5, 8]), c([0, 4, 8]))
    _ok()
    outside = torch.tensor([True, True, *[False] * 6, True, True]).cuda()
    assert not out[outside].any() and (lse[outside] == -float("inf")).all() and torch.isfinite(lse[~outside]).all()
    out, lse = call(c([0, 12]), c([0, 11]))  # past the tensors: clamped and recorded
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_ERR_DEVICE and torch.isfinite(out.float()).all()
    out, lse = csa.sparse_attn_forward(q.cuda(), k.cuda(), v.cuda(), idx.cuda(), c([0]), c([0]), 0.125)
    _ok()
    assert not out.any() and (lse == -float("inf")).all()


# ----------------------------------------------------------------------------- gradients
@pytest.mark.parametrize("shape", SHAPES, ids=_shape_id)
@pytest.mark.parametrize("lengths", LENGTHS)
def test_gradients(lengths, shape):
    lq, lk = LENGTHS[lengths]
    Hq, Hk, D, dt, K, block, window = shape
    q, k, v, do = _inputs(lq, lk, Hq, Hk, D, dt, seed=len(lq) + D)
    idx = _lists(lq, lk, K, block, seed=K)
    _run(q, k, v, do, idx, _cu(lq), _cu(lk), D ** -0.5, block=block, window=window)


@pytest.mark.parametrize("Hq,Hk,D,dt", [(64, 1, 128, BF), (96, 1, 64, FP16), (134, 2, 64, BF), (8, 8, 128, FP16)])
def test_gradients_without_causal_border_and_odd_groups(Hq, Hk, D, dt):
    lq, lk = [40, 0, 3, 61, 1], [129, 3, 257, 40, 0]
    q, k, v, do = _inputs(lq, lk, Hq, Hk, D, dt, seed=Hq)
    idx = _lists(lq, lk, 50, 2, seed=5)
    _run(q, k, v, do, idx, _cu(lq), _cu(lk), D ** -0.5, block=2, causal=False)


def test_gradients_of_a_window_alone():
    lq = [70, 1, 300]
    q, k, v, do = _inputs(lq, lq, 4, 2, 64, BF, seed=9)
    _run(q, k, v, do, None, _cu(lq), _cu(lq), 0.125, window=50)
    _run(q, k, v, do, None, _cu(lq), _cu(lq), 0.125, window=1000)


def test_gradients_of_a_key_that_every_row_lists():
    T = 1500
    q, k, v, do = _inputs([T], [300], 4, 1, 64, BF, seed=20)
    idx = _lists([T], [300], 9, 1, seed=6, holes=0.0)
    idx[:, 0] = torch.where((idx[:, 1:] == 7).any(1), -1, 7)
    _run(q, k, v, do, idx, _cu([T]), _cu([300]), 0.125, causal=False)


@pytest.mark.parametrize("N", [31, 32, 75])
def test_gradients_of_many_sequences(N):
    # up to 31 are held by the lanes, more are searched; lengths of zero to 13 rows, so no row's sequence is guessed
    rng = np.random.default_rng(N)
    lq = rng.integers(0, 14, N).tolist()
    lk = [n + int(m) for n, m in zip(lq, rng.integers(0, 60, N))]
    q, k, v, do = _inputs(lq, lk, 6, 2, 64, BF, seed=25)
    idx = _lists(lq, lk, 11, 2, seed=12)
    out = _run(q, k, v, do, idx, _cu(lq), _cu(lk), 0.125, block=2, window=7)
    # the same keys in pages, in another order
    page, width = 8, -(-max(lk) // 8)
    table = torch.randperm(N * width, generator=torch.Generator().manual_seed(1)).reshape(N, width).to(torch.int32)
    kp, vp = (torch.full((N * width, page, 2, 64), float("nan"), dtype=BF) for _ in range(2))
    at = 0
    for i, n in enumerate(lk):
        for j in range(n):
            kp[table[i, j // page], j % page], vp[table[i, j // page], j % page] = k[at + j], v[at + j]
        at += n
    c = lambda t: t.cuda()  # noqa: E731
    paged = csa.sparse_attn_paged(c(q), c(kp), c(vp), c(table), c(idx), c(_cu(lq)), torch.tensor(lk, dtype=torch.int32).cuda(),
                                  0.125, block=2, window=7)
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(paged, out))


def test_gradients_where_blocks_are_many():
    # 90003 numbers of blocks: the running sum of the lists takes 22 steps, and groups have several rows
    lq, lk = [450, 0, 150], [50000, 3, 39997]
    q, k, v, do = _inputs(lq, lk, 2, 1, 64, BF, seed=24)
    idx = _lists(lq, lk, 40, 1, seed=11)
    idx[::3, 5] = 4095 + torch.arange(200, dtype=torch.int32) % 3  # keys with many rows, at the border of a step
    idx[:, 6:][(idx[:, 6:] >= 4095) & (idx[:, 6:] <= 4097)] = -1
    idx[:, :5][(idx[:, :5] >= 4095) & (idx[:, :5] <= 4097)] = -1
    _run(q, k, v, do, idx, _cu(lq), _cu(lk), 0.125, causal=False)


def test_gradients_of_a_block_listed_twice():
    q, k, v, do = _inputs([3], [40], 4, 2, 64, BF, seed=4)
    idx = torch.tensor([[3, 3, 1, -1], [0, 2, 0, 0], [5, 5, 5, 5]], dtype=torch.int32)
    _run(q, k, v, do, idx, _cu([3]), _cu([40]), 0.2, block=4, causal=False)


def test_gradients_with_lengths_of_keys():
    lq, lk = [6, 30], [200, 100]
    q, k, v, do = _inputs(lq, lk, 8, 2, 128, FP16, seed=6)
    k_len = torch.tensor([150, 31], dtype=torch.int32)
    idx = _lists(lq, [150, 31], 20, 2, seed=1)
    r = _run(q, k, v, do, idx, _cu(lq), _cu(lk), 0.1, k_len=k_len, block=2, window=9)
    past = torch.tensor([*range(150, 200), *range(231, 300)]).cuda()
    assert not r[3][past].any() and not r[4][past].any()
    k[past.cpu()], v[past.cpu()] = float("nan"), float("inf")
    c = lambda t: t.cuda()  # noqa: E731
    again = csa.sparse_attn_backward(c(do), c(q), c(k), c(v), r[0], r[1], c(idx), c(_cu(lq)), c(_cu(lk)), 0.1, k_len=c(k_len),
                                     block=2, window=9)
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(again, r[2:]))


@pytest.mark.parametrize("size", [1.0, 2.0 ** 14, 2.0 ** -12])
def test_gradients_of_scaled_cotangents_fp16(size):
    lq = [90, 33]
    q, k, v, do = _inputs(lq, lq, 6, 2, 64, FP16, seed=22)
    do = (do.float() * size).clamp(-60000, 60000).to(FP16)
    if size > 1:  # gradients that fit fp16 of weights and differences that do not
        v = (v.float() * 2.0 ** -8).to(FP16)
        q, k = ((t.float() * 2.0 ** -5).to(FP16) for t in (q, k))
        do = (do.float() * 2.0 ** -5).to(FP16)
    idx = _lists(lq, lq, 12, 4, seed=8)
    _run(q, k, v, do, idx, _cu(lq), _cu(lq), 0.125, block=4, window=3)


def test_gradients_in_several_rounds_repeat_bit_for_bit():
    # 6 GB of shares: two rounds; lists of all rows in a different order of places give the same sums only if the
    # order of the sums is that of the rows
    T, W, Hk, K = 1500, 1100, 8, 1024
    q, k, v, do = _inputs([T], [W], Hk, Hk, 128, BF, seed=23)
    idx = _lists([T], [W], K, 1, seed=9, holes=0.1)
    one = _run(q, k, v, do, idx, _cu([T]), _cu([W]), 128 ** -0.5, causal=False)
    c = lambda t: t.cuda()  # noqa: E731
    two = csa.sparse_attn_backward(c(do), c(q), c(k), c(v), one[0], one[1], c(idx), c(_cu([T])), c(_cu([W])), 128 ** -0.5,
                                   causal=False)
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(one[2:], two))


def test_gradients_against_differences():
    """Along a direction e of one input, with the forward in 64 bits: (L(x + h e) - L(x - h e)) / 2h = sum g e.  The
    kernel's g is off by at most the bounds of _bounds, whose magnitudes are summed here with |e|."""
    lq, lk = [20, 7], [60, 30]
    q, k, v, do = _inputs(lq, lk, 8, 2, 64, BF, seed=24)
    idx = _lists(lq, lk, 9, 2, seed=10)
    kw = dict(block=2, window=4)
    r = _run(q, k, v, do, idx, _cu(lq), _cu(lk), 0.125, **kw)
    a = (idx.numpy(), _cu(lq).numpy(), _cu(lk).numpy(), 0.125)
    x = [f64(t) for t in (q, k, v)]
    ref = S.attention(*x, *a, **kw, dout=f64(do))
    b = _bounds(ref, BF)
    rng = np.random.default_rng(0)
    loss = lambda x: (S.attention(*x, *a, **kw)["out"] * f64(do)).sum()  # noqa: E731
    for i, name in enumerate(("dq", "dk", "dv")):
        e = rng.standard_normal(x[i].shape)
        up, down = ([t + s * 1e-5 * e if n == i else t for n, t in enumerate(x)] for s in (1, -1))
        want = (loss(up) - loss(down)) / 2e-5
        assert abs((f64(r[2 + i]) * e).sum() - want) <= (b[name] * np.abs(e)).sum() + 1e-6


def test_gradients_do_not_leak_and_replay_from_a_graph():
    lq = [50, 37, 64]
    q, k, v, do = (t.cuda() for t in _inputs(lq, lq, 8, 2, 128, BF, seed=25))
    idx, cu = _lists(lq, lq, 10, 4, seed=11).cuda(), _cu(lq).cuda()

    def both():
        out, lse = csa.sparse_attn_forward(q, k, v, idx, cu, cu, 0.1, block=4, window=6)
        return (out, lse, *csa.sparse_attn_backward(do, q, k, v, out, lse, idx, cu, cu, 0.1, block=4, window=6))

    want = [t.clone() for t in both()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both()
    for _ in range(2):
        g.replay()
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for t in (q, k, v, do):
        t[50:87] = float("nan")
    other = torch.tensor([*range(50), *range(87, 151)]).cuda()
    assert all(torch.equal(a[other], b[other]) for a, b in zip(both(), want))
    _ok()


def test_gradients_without_keys_or_rows():
    q, k, v, do = (t.cuda() for t in _inputs([5], [7], 4, 2, 64, FP16, seed=26))
    c = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    idx = torch.zeros(5, 2, dtype=torch.int32).cuda()
    none = k[:0]
    out, lse = csa.sparse_attn_forward(q, none, none, idx - 1, c([0, 5]), c([0, 0]), 0.1)
    g = csa.sparse_attn_backward(do, q, none, none, out, lse, idx - 1, c([0, 5]), c([0, 0]), 0.1)
    assert not out.any() and not g[0].any() and g[1].shape == none.shape
    e = q[:0]
    g = csa.sparse_attn_backward(e, e, k, v, e, lse[:0], idx[:0], c([0, 0]), c([0, 7]), 0.1)
    assert not g[1].any() and not g[2].any()
    g = csa.sparse_attn_backward(do, q, k, v, torch.zeros_like(q), torch.full_like(lse, -float("inf")), idx, c([0]), c([0]), 0.1)
    assert not any(t.any() for t in g)
    _ok()


# ----------------------------------------------------------------------------- paged
def _paged(k, v, lk, page, seed=0, spare=2):
    """A shuffled pool holding packed k, v, its table; the rest of the pool is NaN."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lk]
    order = rng.permutation(sum(need) + spare)
    pool = [torch.full((len(order), page, *k.shape[1:]), float("nan"), dtype=k.dtype) for _ in range(2)]
    table = np.full((len(lk), max(need) + 1), -1, dtype=np.int32)
    at = c = 0
    for i, n in enumerate(lk):
        table[i, :need[i]] = order[at:at + need[i]]
        for j in range(n):
            for p, x in zip(pool, (k, v)):
                p[table[i, j // page], j % page] = x[c + j]
        at, c = at + need[i], c + n
    return *pool, torch.tensor(table)


@pytest.mark.parametrize("page", [1, 24, 64, 100])
@pytest.mark.parametrize("lq,lk", [([1, 1, 1], [300, 1, 129]), ([3, 0, 5], [200, 40, 4])], ids=str)
def test_paged_gives_the_packed_bits(page, lq, lk):
    for Hq, Hk, D, dt in ((8, 2, 128, BF), (5, 1, 64, FP16)):
        q, k, v, _ = _inputs(lq, lk, Hq, Hk, D, dt, seed=page)
        idx = _lists(lq, lk, 20, 4, seed=page)
        kp, vp, table = _paged(k, v, lk, page)
        c = lambda t: t.cuda()  # noqa: E731
        kw = dict(block=4, window=13)
        want = csa.sparse_attn_forward(c(q), c(k), c(v), c(idx), c(_cu(lq)), c(_cu(lk)), 0.1, **kw)
        k_len = torch.tensor(lk, dtype=torch.int32).cuda()
        got = csa.sparse_attn_paged(c(q), c(kp), c(vp), c(table), c(idx), c(_cu(lq)), k_len, 0.1, **kw)
        # keys and values side by side in one pool, the table a view
        both = torch.stack([kp, vp], 1).cuda()
        wide = torch.cat([table, table], 1).cuda()
        two = csa.sparse_attn_paged(c(q), both[:, 0], both[:, 1], wide[:, :table.shape[1]], c(idx), c(_cu(lq)), k_len,
                                    0.1, **kw)
        _ok()
        assert all(torch.equal(a, b) and torch.equal(a, d) for a, b, d in zip(want, got, two))


def test_bad_pages_are_reported_and_skipped():
    lq, lk = [1, 2], [40, 33]
    q, k, v, _ = _inputs(lq, lk, 4, 2, 64, BF, seed=15)
    kp, vp, table = _paged(k, v, lk, 8)
    idx = _lists(lq, lk, 10, 8, seed=4, holes=0.0)
    k_len = torch.tensor(lk, dtype=torch.int32).cuda()
    call = lambda i, t, n=k_len: csa.sparse_attn_paged(q.cuda(), kp.cuda(), vp.cuda(), t.cuda(), i.cuda(),  # noqa: E731
                                                       _cu(lq).cuda(), n, 0.1, block=8)
    less = idx.clone()
    less[0][less[0] == 1] = -1
    want = call(less, table)
    _ok()
    for value in (-1, kp.shape[0], 2 ** 31 - 1):
        bad = table.clone()
        bad[0, 1] = value
        got = call(idx, bad)
        torch.cuda.synchronize()
        assert csa.device_status() == csa.CSA_ERR_DEVICE
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    call(idx, table, k_len + 1000)  # longer than the table: clamped and recorded
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_ERR_DEVICE


def test_two_replayed_graphs_and_another_stream():
    lq, lk = [1] * 4, [700] * 4
    q, k, v, _ = (t.cuda() for t in _inputs(lq, lk, 16, 2, 128, BF, seed=16))
    idx = _lists(lq, lk, 60, 8, seed=5).cuda()
    cu_q, cu_k = _cu(lq).cuda(), _cu(lk).cuda()
    call = lambda q, **kw: csa.sparse_attn_forward(q, k, v, idx, cu_q, cu_k, 0.1, block=8, window=20, **kw)  # noqa: E731
    q2 = q.flip(0).contiguous()
    want, want2 = call(q), call(q2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(q, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs, x = [], [], [q.clone(), q2.clone()]
    for t in x:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(t))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(want, outs[0])) and all(torch.equal(a, b) for a, b in zip(want2, outs[1]))
    x[0].copy_(q2)
    graphs[0].replay()
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(want2, outs[0]))
