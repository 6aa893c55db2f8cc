"""Packed attention on the GPU against the fp64 definition, forward and gradients.

Tolerances, from the arithmetic (u = eps/2 of the storage type):
* scores: products of stored values are exact in fp32 and up to 128 of them are
  added in fp32, with two more roundings for the scale: an error ds of at most
  2^-16 of the row's largest scale*|q|.|k|.
* p = exp(s - m) therefore is off by ds relative, 2^-20 for the exponential, and
  u where it is rounded to the storage type for the product with v; the sum
  (fp32, of unrounded p) by the same but u.  fp16 cannot hold p below 2^-24: at
  most 2^-25 absolute per key.  out is rounded once.
      |out - ref| <= u |ref| + (u + 2 ds + 2^-18) sum p|v| + 2^-25 sum |v|
      |lse - ref| <= ds + 2^-19 + 2^-22 |ref|
* gradients: p as above; ds = p (dout.v - delta) is rounded to the storage type,
  delta = dout.out uses the rounded out (u sum|dout||out|), dout.v is a fp32 sum
  (2^-16 |dout|.|v|).  With mag the sum of |ds| + p (sum|dout||out| + |dout|.|v|)
  over the terms, times the other factor:
      |dq - ref| <= u |ref| + (2u + 2 ds + 2^-15) mag + 2^-25 (sum of the other factor)
  and the same for dk; dv has u + 2 ds + 2^-18.
  The 2^-25 terms are for fp16 alone (bf16 has fp32's range).
"""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from oracle import attn_oracle as A

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


def _check(name, got, want, bound):
    g = A.f64(got)
    assert np.array_equal(np.isneginf(g), np.isneginf(want)), name
    fin = ~np.isneginf(want)
    assert np.isfinite(g[fin]).all(), name
    err = np.abs(np.where(fin, g, 0) - np.where(fin, want, 0))
    r = err / (np.where(fin, bound, 1) + 1e-30)
    assert r.max(initial=0.0) <= 1.0, (name, float(r.max()), np.unravel_index(r.argmax(), r.shape))


def _bounds(ref, dt):
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == FP16 else 0.0
    ds = 2.0 ** -16 * ref["smax"]
    lse = np.where(np.isneginf(ref["lse"]), 0, ref["lse"])
    b = dict(out=u * np.abs(ref["out"]) + (u + 2 * ds[..., None] + 2.0 ** -18) * ref["mag_out"] + tiny * ref["vsum"],
             lse=ds + 2.0 ** -19 + 2.0 ** -22 * np.abs(lse))
    top = 2 * ds.max(initial=0.0)
    for n in ("dq", "dk", "dv"):
        if n in ref:
            rel = (u + top + 2.0 ** -18) if n == "dv" else (2 * u + top + 2.0 ** -15)
            b[n] = u * np.abs(ref[n]) + rel * ref["mag_" + n] + tiny * ref["sum_" + n]
    return b


def _run(q, k, v, do, cu_q, cu_k, scale, causal=True, k_len=None, backward=True):
    """Forward and gradients on the GPU, checked against the definition."""
    dt = q.dtype
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    qg, kg, vg, dog, cq, ck, kl = (c(t) for t in (q, k, v, do, cu_q, cu_k, k_len))
    out, lse = csa.attn_forward(qg, kg, vg, cq, ck, scale, causal=causal, k_len=kl)
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK
    n = lambda t: None if t is None else t.numpy()  # noqa: E731
    ref = A.attention(A.f64(q), A.f64(k), A.f64(v), n(cu_q), n(cu_k), scale, causal, n(k_len),
                      A.f64(do) if backward else None)
    b = _bounds(ref, dt)
    _check("out", out, ref["out"], b["out"])
    _check("lse", lse, ref["lse"], b["lse"])
    if backward:
        grads = csa.attn_backward(dog, qg, kg, vg, out, lse, cq, ck, scale, causal=causal, k_len=kl)
        torch.cuda.synchronize()
        assert csa.device_status() == csa.CSA_OK
        for name, t in zip(("dq", "dk", "dv"), grads):
            _check(name, t, ref[name], b[name])
    return out, lse


LENGTHS = {
    "one": ([1], [1]),
    "tile_edges": ([127, 128, 129], [127, 128, 129]),
    "around_32": ([15, 16, 17, 31, 33], [15, 16, 17, 31, 33]),
    "empty_ones": ([0, 5, 0, 0, 70, 0], [0, 5, 9, 0, 70, 0]),
    "no_keys": ([4, 3], [0, 3]),
    "rows_without_keys": ([200, 40, 150], [60, 39, 1]),
    "behind_a_prefix": ([1, 33, 64, 7], [300, 500, 65, 129]),
    "long": ([700], [700]),
    "many": ([3, 1, 2, 40, 9, 1, 1, 1, 17, 5, 130, 8, 1, 66, 2, 257, 4, 6, 90, 10] * 2,
             [3, 1, 2, 40, 9, 1, 1, 1, 17, 5, 130, 8, 1, 66, 2, 257, 4, 6, 90, 10] * 2),
}
HEADS = [(1, 1, 128, BF), (8, 1, 64, FP16), (6, 2, 128, FP16), (12, 4, 64, BF), (16, 2, 128, BF), (7, 7, 64, BF),
         (40, 1, 128, BF)]


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: f"{h[0]}q{h[1]}k_D{h[2]}_{str(h[3])[6:]}")
@pytest.mark.parametrize("lengths", LENGTHS)
def test_against_definition(lengths, heads):
    lq, lk = LENGTHS[lengths]
    Hq, Hk, D, dt = heads
    q, k, v, do = _inputs(lq, lk, Hq, Hk, D, dt, seed=len(lq) + D)
    _run(q, k, v, do, _cu(lq), _cu(lk), D ** -0.5)


@pytest.mark.parametrize("dt,D", [(BF, 128), (FP16, 64)])
def test_without_causal_mask(dt, D):
    lq, lk = [5, 130, 0, 33, 1], [70, 129, 3, 257, 0]
    q, k, v, do = _inputs(lq, lk, 8, 2, D, dt, seed=3)
    _run(q, k, v, do, _cu(lq), _cu(lk), D ** -0.5, causal=False)


@pytest.mark.parametrize("causal", [True, False])
def test_group_of_128_heads_and_odd_group(causal):
    for Hq in (128, 100):
        lq, lk = [3, 9], [40, 9]
        q, k, v, do = _inputs(lq, lk, Hq, 1, 64, BF, seed=Hq)
        _run(q, k, v, do, _cu(lq), _cu(lk), 0.125, causal=causal)


def test_large_scores_and_running_maximum():
    # scores up to several hundred, growing along the keys: every tile raises the running maximum
    q, k, v, do = _inputs([600], [600], 4, 1, 128, BF, seed=8, size=2.0)
    k = (k.float() * torch.linspace(0.1, 4.0, 600)[:, None, None]).to(BF)
    _run(q, k, v, do, _cu([600]), _cu([600]), 1.0, backward=False)
    k = k.flip(0).contiguous()  # and falling: the first tile holds the maximum
    _run(q, k, v, do, _cu([600]), _cu([600]), 1.0, backward=False)


def test_decode_over_a_cache_with_lengths():
    N, W, Hq, Hk, D = 9, 640, 16, 2, 128
    lens = torch.tensor([1, 127, 128, 129, 0, 640, 333, 512, 2], dtype=torch.int32)
    q, k, v, do = _inputs([1] * N, [W] * N, Hq, Hk, D, BF, seed=5)
    cu_k = torch.arange(N + 1, dtype=torch.int32) * W
    _run(q, k, v, do, _cu([1] * N), cu_k, D ** -0.5, k_len=lens)
    # what the cache holds past the lengths is not part of the result
    c = lambda t: t.cuda()  # noqa: E731
    args = (c(_cu([1] * N)), c(cu_k), D ** -0.5)
    one = csa.attn_forward(c(q), c(k), c(v), *args, k_len=c(lens))
    past = (torch.arange(W)[None] >= lens[:, None]).reshape(-1)
    for bad in (float("nan"), float("inf"), -float("inf")):
        k[past], v[past] = bad, bad
        two = csa.attn_forward(c(q), c(k), c(v), *args, k_len=c(lens))
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        grads = csa.attn_backward(c(do), c(q), c(k), c(v), *one, *args, k_len=c(lens))
        assert all(torch.isfinite(g).all() for g in grads)
        assert not grads[1][past.cuda()].any() and not grads[2][past.cuda()].any()


@pytest.mark.parametrize("N,W,Hq,Hk,D,dt", [(1, 9000, 8, 1, 128, BF), (3, 5000, 6, 2, 64, FP16), (2, 20001, 4, 4, 128, BF)])
def test_long_caches(N, W, Hq, Hk, D, dt):
    # few rows, many keys
    lens = torch.randint(W // 2, W + 1, (N,), generator=torch.Generator().manual_seed(W), dtype=torch.int32)
    lens[0] = W
    q, k, v, do = _inputs([1] * N, [W] * N, Hq, Hk, D, dt, seed=W)
    _run(q, k, v, do, _cu([1] * N), torch.arange(N + 1, dtype=torch.int32) * W, D ** -0.5, k_len=lens, backward=False)


def test_few_rows_over_a_long_prefix():
    # speculative or chunked decoding: several rows per sequence, the split keys end in the causal border
    lq, lk = [5, 40, 3], [3001, 2100, 2]
    q, k, v, do = _inputs(lq, lk, 8, 2, 128, BF, seed=21)
    _run(q, k, v, do, _cu(lq), _cu(lk), 128 ** -0.5)


def test_other_sequences_do_not_leak():
    # NaN in one sequence's rows, keys and values leaves the others' bits alone
    lq = [100, 37, 130, 60]
    q, k, v, do = _inputs(lq, lq, 8, 2, 128, BF, seed=6)
    cu = _cu(lq)
    c = lambda t: t.cuda()  # noqa: E731

    def both():
        o = csa.attn_forward(c(q), c(k), c(v), c(cu), c(cu), 0.1)
        return (*o, *csa.attn_backward(c(do), c(q), c(k), c(v), *o, c(cu), c(cu), 0.1))

    good = both()
    bad_rows = torch.zeros(sum(lq), dtype=torch.bool)
    bad_rows[100:137] = True
    for t in (q, k, v, do):
        t[bad_rows] = float("nan")
    for a, b in zip(good, both()):
        assert torch.equal(a[~bad_rows.cuda()], b[~bad_rows.cuda()])


@pytest.mark.parametrize("lq,lk,Hq,Hk,D,dt", [([200], [200], 8, 1, 128, BF), ([300, 40], [300, 90], 4, 4, 64, FP16),
                                              ([24], [5000], 8, 1, 128, BF), ([3], [700], 6, 2, 64, FP16)])
def test_hidden_keys_of_the_sequence_do_not_leak(lq, lk, Hq, Hk, D, dt):
    """Infinite and NaN keys and values reach the rows that see them and no others."""
    q, k, v, _ = _inputs(lq, lk, Hq, Hk, D, dt, seed=31)
    cu_q, cu_k = _cu(lq).cuda(), _cu(lk).cuda()
    run = lambda: csa.attn_forward(q.cuda(), k.cuda(), v.cuda(), cu_q, cu_k, D ** -0.5)  # noqa: E731
    good, good_lse = run()
    first = lk[0] - lq[0]                 # the last key that row 0 sees
    at = first + lq[0] // 2               # seen from row lq/2 on
    rows = lq[0] // 2
    v[at, 0, 3], v[at, 0, 5], v[at, 0, 60] = float("inf"), -float("inf"), float("nan")
    v[lk[0] - 1, Hk - 1, 7] = float("nan")   # seen by the last row alone
    out, lse = run()
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK
    assert torch.equal(lse, good_lse)
    g = Hq // Hk
    changed = torch.zeros_like(out, dtype=torch.bool)
    changed[rows:lq[0], :g, 3] = changed[rows:lq[0], :g, 5] = changed[rows:lq[0], :g, 60] = True
    changed[lq[0] - 1, Hq - g:, 7] = True
    assert torch.equal(out[~changed], good[~changed])
    assert (out[rows:lq[0], :g, 3] == float("inf")).all() and (out[rows:lq[0], :g, 5] == -float("inf")).all()
    assert out[rows:lq[0], :g, 60].isnan().all() and out[lq[0] - 1, Hq - g:, 7].isnan().all()
    # a NaN key: the rows that see it are NaN, the others keep their bits
    k[lk[0] - 1, 0, 0] = float("nan")
    out2, lse2 = run()
    same = torch.ones(sum(lq), Hq, dtype=torch.bool, device="cuda")
    same[lq[0] - 1, :g] = False
    assert torch.equal(lse2[same], good_lse[same]) and lse2[~same].isnan().all() and out2[lq[0] - 1, :g].isnan().all()
    assert torch.equal(out2[same].nan_to_num(3.0), out[same].nan_to_num(3.0))


def test_rows_outside_every_sequence():
    q, k, v, do = _inputs([50], [60], 4, 2, 64, BF, seed=7)
    cu_q, cu_k = torch.tensor([10, 30, 41], dtype=torch.int32), torch.tensor([5, 20, 51], dtype=torch.int32)
    out, lse = _run(q, k, v, do, cu_q, cu_k, 0.125)
    assert not out[:10].any() and not out[41:].any() and torch.isneginf(lse[:10]).all() and torch.isneginf(lse[41:]).all()


def test_no_sequences_and_no_rows():
    q, k, v, do = (t.cuda() for t in _inputs([5], [6], 4, 2, 64, BF))
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = csa.attn_forward(q, k, v, none, none, 0.1)
    assert not out.any() and torch.isneginf(lse).all()
    assert not any(g.any() for g in csa.attn_backward(do, q, k, v, out, lse, none, none, 0.1))
    e = q[:0].contiguous()
    cu0, cu6 = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    out, lse = csa.attn_forward(e, k, v, cu0, cu6, 0.1)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    dq, dk, dv = csa.attn_backward(e, e, k, v, out, lse, cu0, cu6, 0.1)
    assert dq.shape == e.shape and not dk.any() and not dv.any()


def test_strided_views():
    # q, k and v as views of one projection's output, and heads further apart than D
    gen = torch.Generator().manual_seed(2)
    lq = [90, 41]
    T, Hq, Hk, D = sum(lq), 6, 2, 64
    wide = torch.randn(T, Hq + 2 * Hk, D + 16, generator=gen).to(BF)
    do = torch.randn(T, Hq, D, generator=gen).to(BF)
    q, k, v = wide[:, :Hq, :D], wide[:, Hq:Hq + Hk, 16:], wide[:, Hq + Hk:, 8:8 + D]
    wg = wide.cuda()
    cu = _cu(lq)
    cg = cu.cuda()
    args = (wg[:, :Hq, :D], wg[:, Hq:Hq + Hk, 16:], wg[:, Hq + Hk:, 8:8 + D])
    out, lse = csa.attn_forward(*args, cg, cg, 0.125)
    grads = csa.attn_backward(do.cuda(), *args, out, lse, cg, cg, 0.125)
    ref = A.attention(A.f64(q), A.f64(k), A.f64(v), cu.numpy(), cu.numpy(), 0.125, dout=A.f64(do))
    b = _bounds(ref, BF)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        _check(name, t, ref[name], b[name])


def test_offsets_past_32_bits():
    # a cache whose last sequence starts beyond 2^32 elements
    W, Hk, D, N = 300_000, 8, 128, 15
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB of device memory")
    cache = torch.empty(N * W, Hk, D, dtype=BF, device="cuda")
    cache2 = torch.empty(N * W, Hk, D, dtype=BF, device="cuda")
    q, k, v, _ = _inputs([1], [700], 16, 8, 128, BF, seed=12)
    at = (N - 1) * W
    assert at * Hk * D > 1 << 32
    cache[at:at + 700], cache2[at:at + 700] = k.cuda(), v.cuda()
    lens = torch.zeros(N, dtype=torch.int32)
    lens[-1] = 700
    qs = torch.zeros(N, 16, 128, dtype=BF)
    qs[-1] = q[0]
    out, lse = csa.attn_forward(qs.cuda(), cache, cache2, torch.arange(N + 1, dtype=torch.int32).cuda(),
                                (torch.arange(N + 1, dtype=torch.int32) * W).cuda(), 128 ** -0.5, k_len=lens.cuda())
    ref = A.attention(A.f64(q), A.f64(k), A.f64(v), [0, 1], [0, 700], 128 ** -0.5)
    b = _bounds(ref, BF)
    _check("out", out[-1:], ref["out"], b["out"])
    _check("lse", lse[-1:], ref["lse"], b["lse"])
    assert not out[:-1].any()


def test_bad_offsets_are_clamped_and_reported():
    q, k, v, do = (t.cuda() for t in _inputs([40], [40], 4, 2, 64, BF))
    ok = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    for bad in ([0, 41], [-3, 40], [30, 10]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for a, b in ((cu, ok), (ok, cu)):
            out, lse = csa.attn_forward(q, k, v, a, b, 0.1)
            assert csa.device_status() == csa.CSA_ERR_DEVICE
            csa.attn_backward(do, q, k, v, out, lse, a, b, 0.1)
            assert csa.device_status() == csa.CSA_ERR_DEVICE
    csa.attn_forward(q, k, v, ok, ok, 0.1, k_len=torch.tensor([41], dtype=torch.int32, device="cuda"))
    assert csa.device_status() == csa.CSA_ERR_DEVICE
    csa.attn_forward(q, k, v, ok, ok, 0.1)
    assert csa.device_status() == csa.CSA_OK


def test_results_repeat_bit_for_bit_on_streams_and_in_graphs():
    lq = [300, 77, 513]
    q, k, v, do = (t.cuda() for t in _inputs(lq, lq, 8, 2, 128, BF, seed=13))
    cu = _cu(lq).cuda()

    def step(stream=None):
        o = csa.attn_forward(q, k, v, cu, cu, 0.1, stream=stream)
        return (*o, *csa.attn_backward(do, q, k, v, *o, cu, cu, 0.1, stream=stream))

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = step(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, cap))


def test_gradient_by_differences():
    # directional difference of sum(out * g): fp16 inputs moved by exact steps
    lq = [30, 21]
    q, k, v, g = _inputs(lq, lq, 4, 2, 64, FP16, seed=17)
    cu = _cu(lq).cuda()
    gen = torch.Generator().manual_seed(18)
    dirs = [torch.randint(-1, 2, t.shape, generator=gen).to(FP16) for t in (q, k, v)]
    h = 2.0 ** -5
    # a step of h from values on a grid of h/4 below 8 is exact in fp16
    q, k, v = ((t.float().clamp(-7, 7) * 128).round() / 128 for t in (q, k, v))

    def value(s):
        a = [(t + s * h * d.float()).to(FP16).cuda() for t, d in zip((q, k, v), dirs)]
        out, _ = csa.attn_forward(*a, cu, cu, 0.125)
        return float((out.double().cpu() * g.double()).sum())

    base = [t.to(FP16).cuda() for t in (q, k, v)]
    out, lse = csa.attn_forward(*base, cu, cu, 0.125)
    grads = csa.attn_backward(g.cuda(), *base, out, lse, cu, cu, 0.125)
    want = sum(float((x.double().cpu() * d.double()).sum()) for x, d in zip(grads, dirs))
    # out is rounded to 2^-11 of values below 4 at independent points: 2^-10 * |g| summed in quadrature, over 2h,
    # six sigma; the curvature's h^2 term is below a tenth of the slope's own size
    noise = 6 * float(g.double().norm()) * 2.0 ** -10 / (2 * h)
    size = sum(float((x.double().cpu().abs() * d.double().abs()).sum()) for x, d in zip(grads, dirs))
    assert abs((value(1) - value(-1)) / (2 * h) - want) <= noise + 0.05 * size


def test_binding_refuses():
    q = torch.zeros(4, 4, 64, dtype=BF, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for a in ((q, q.half(), q, cu, cu), (q, q, q[:3], cu, cu), (q, q, q, cu.long(), cu), (q, q, q, cu, cu[:1]),
              (q.transpose(0, 2), q, q, cu, cu), (q, q[:, :1].expand(4, 3, 64), q[:, :1].expand(4, 3, 64), cu, cu)):
        with pytest.raises((ValueError, csa.CsaError)):
            csa.attn_forward(*a, 0.1)
    with pytest.raises(csa.CsaError):
        csa.attn_forward(q.float(), q.float(), q.float(), cu, cu, 0.1)
    with pytest.raises(ValueError):
        csa.attn_forward(q, q, q, cu, cu, 0.1, k_len=cu)
