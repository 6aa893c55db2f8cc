"""Gradients of attention over listed blocks where scales, magnitudes or hidden values are extreme, and where the
softmax spans the keys of two calls.

Tolerances are those of test_gpu_sparse (its docstring derives them); they scale with the inputs.
"""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from oracle import sparse_oracle as S
from oracle.attn_oracle import f64
from test_gpu_sparse import BF, FP16, _cu, _inputs, _lists, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    csa.load()


@pytest.mark.parametrize("dt", [BF, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hk,K", [(1, 1, 20), (6, 2, 20), (64, 1, 150)])
@pytest.mark.parametrize("scale", [8.0, 32.0])
def test_gradients_at_large_scales(scale, Hq, Hk, K, dt):
    """Scores spread over hundreds of nats, so that most weights are zero, and every third row has no cotangent: the
    shares of such keys are zero whatever the scale."""
    lq, lk = [30, 9], [200, 31]
    q, k, v, do = _inputs(lq, lk, Hq, Hk, 128, dt, seed=31)
    do[::3] = 0
    idx = _lists(lq, lk, K, 1, seed=13)
    _run(q, k, v, do, idx, _cu(lq), _cu(lk), scale, causal=False)


def test_gradients_at_a_scale_that_small_queries_and_keys_bring_down():
    lq, lk = [30, 9], [200, 31]
    q, k, v, do = _inputs(lq, lk, 6, 2, 64, BF, seed=32)
    q, k = ((t.float() * 2.0 ** -45).to(BF) for t in (q, k))
    do[::3] = 0
    _run(q, k, v, do, _lists(lq, lk, 20, 1, seed=14), _cu(lq), _cu(lk), 2.0 ** 87, causal=False)


@pytest.mark.parametrize("size", [2.0 ** -80, 2.0 ** -90, 2.0 ** 66, 2.0 ** 90])
@pytest.mark.parametrize("Hq,Hk,K", [(6, 2, 20), (64, 1, 150)])
def test_gradients_of_tiny_and_huge_cotangents(Hq, Hk, K, size):
    """Cotangents whose squares leave fp32's range: dv, dk and dq are of the cotangents' size."""
    lq, lk = [30, 9], [200, 31]
    q, k, v, do = _inputs(lq, lk, Hq, Hk, 128, BF, seed=33)
    do = (do.float() * size).to(BF)
    do[::5] = 0
    _run(q, k, v, do, _lists(lq, lk, K, 1, seed=15), _cu(lq), _cu(lk), 128 ** -0.5, causal=False)


@pytest.mark.parametrize("size", [2.0 ** -80, 2.0 ** 66])
def test_gradients_of_tiny_and_huge_queries(size):
    lq, lk = [30, 9], [200, 31]
    q, k, v, do = _inputs(lq, lk, 6, 2, 64, BF, seed=34)
    q = (q.float() * size).to(BF)
    if size > 1:
        k = (k.float() / size).to(BF)
    _run(q, k, v, do, _lists(lq, lk, 20, 1, seed=16), _cu(lq), _cu(lk), 0.125, causal=False)


def test_gradients_of_rows_of_many_sizes():
    lq, lk = [60], [90]
    q, k, v, do = _inputs(lq, lk, 4, 1, 64, BF, seed=35)
    do = (do.float() * (2.0 ** torch.arange(-100, 80, 3.0))[:60, None, None]).to(BF)
    idx = torch.arange(60, dtype=torch.int32)[:, None]  # a key has the rows of one size
    _run(q, k, v, do, idx, _cu(lq), _cu(lk), 0.125, causal=False)


@pytest.mark.parametrize("Hq,Hk,K", [(6, 2, 20), (64, 1, 150)])
def test_gradients_up_to_the_end_of_the_range(Hq, Hk, K):
    """dk and dv above 2^110."""
    lq, lk = [30, 9], [200, 31]
    q, k, v, do = _inputs(lq, lk, Hq, Hk, 64, BF, seed=36)
    do = (do.float() * 2.0 ** 112).to(BF)
    v = (v.float() * 2.0 ** -4).to(BF)
    r = _run(q, k, v, do, _lists(lq, lk, K, 1, seed=17), _cu(lq), _cu(lk), 0.125, causal=False)
    assert r[4].abs().max() > 2.0 ** 111


@pytest.mark.parametrize("paths", [(6, 2, 64, 20, 2, 9), (64, 1, 128, 150, 1, 0), (40, 1, 64, 0, 1, 33)],
                         ids=["one_tile", "several_tiles", "window"])
@pytest.mark.parametrize("dt", [BF, FP16], ids=["bf16", "fp16"])
def test_gradients_do_not_depend_on_values_that_a_row_does_not_see(paths, dt):
    """Finite large values, infinities and NaN at keys that no row sees, and at one that a single row sees: the other
    rows' dq and the other keys' dk and dv keep their bits."""
    Hq, Hk, D, K, block, window = paths
    lq, lk = [30, 9], [400, 90]
    q, k, v, do = (t.cuda() for t in _inputs(lq, lk, Hq, Hk, D, dt, seed=37))
    idx = None
    if K:
        idx = _lists(lq, [n - 60 for n in lk], K, block, seed=18)
        first = idx[:30]
        first[first == 5] = -1  # of the first sequence only row 7 lists block 5
        first[7, 0] = 5
        first[7, 1:][first[7, 1:] == 5] = -1
    cq, ck = _cu(lq), _cu(lk)
    lists = np.zeros((39, 0), dtype=np.int32) if idx is None else idx.numpy()
    n = [S.counts(lists[a:b], np.arange(b - a) + m - (b - a), m, block, window, window > 0)
         for a, b, m in ((0, 30, 400), (30, 39, 90))]
    seen = np.concatenate([x.any(0) for x in n])
    assert (~seen).sum() > 50
    if idx is not None:
        idx = idx.cuda()
    kw = dict(block=block, window=window, causal=window > 0)

    def grads(k, v):
        out, lse = csa.sparse_attn_forward(q, k, v, idx, cq.cuda(), ck.cuda(), 0.1, **kw)
        g = csa.sparse_attn_backward(do, q, k, v, out, lse, idx, cq.cuda(), ck.cuda(), 0.1, **kw)
        torch.cuda.synchronize()
        assert csa.device_status() == csa.CSA_OK
        return g

    want = grads(k, v)
    hidden = torch.tensor(~seen).cuda()
    for bad in (6e4, float("inf"), float("nan")):
        k2, v2 = k.clone(), v.clone()
        k2[hidden], v2[hidden] = bad, bad
        assert all(torch.equal(a, b) for a, b in zip(grads(k2, v2), want)), bad
    # a key that few rows see
    key = int(np.argmin(np.where(n[0].any(0), n[0].sum(0), 99)))
    rows = torch.zeros(39, dtype=torch.bool)
    rows[:30] = torch.tensor(n[0][:, key] > 0)
    keys = torch.zeros(490, dtype=torch.bool)
    keys[:400] = torch.tensor(n[0][rows[:30].numpy()].any(0))
    assert 0 < rows.sum() < 30 and 0 < keys.sum() < seen.sum()
    v2 = v.clone()
    v2[key] = 6e4
    got = grads(k, v2)
    rows, keys = rows.cuda(), keys.cuda()
    assert torch.equal(got[0][~rows], want[0][~rows])
    assert torch.equal(got[1][~keys], want[1][~keys]) and torch.equal(got[2][~keys], want[2][~keys])


def masked(q, k, v, do, out, lse, see, scale, dt, shares=True):
    """Gradients in 64 bits of a call whose rows see the keys `see` [rows,keys] (one sequence), as a part of a softmax
    whose out and lse are given: p = exp(s - lse), ds = p (dp - dout.out).  With their bounds, those of test_gpu_sparse:
    u |ref| + (2u + 2 ds + 2^-15 of the magnitudes), the shares' 2^-11 and 2^-39, fp16's spacing (ds is bounded by
    |dout| max|v| + |dout.out| too, as out may hold other calls' values)."""
    u = torch.finfo(dt).eps / 2
    h = 1.0 if dt == FP16 else 0.0
    sh = 1.0 if shares and dt != FP16 else 0.0
    Q, K, V, G, O, L = (f64(t) for t in (q, k, v, do, out, lse))
    g = Q.shape[1] // K.shape[1]
    val = {n: np.zeros(x.shape) for n, x in (("dq", Q), ("dk", K), ("dv", V))}
    err = {n: np.zeros(x.shape) for n, x in (("dq", Q), ("dk", K), ("dv", V))}
    for x in range(Q.shape[1]):
        j = x // g
        s = scale * Q[:, x] @ K[:, j].T
        ds = 2.0 ** -16 * np.where(see, scale * np.abs(Q[:, x]) @ np.abs(K[:, j]).T, 0).max(1, keepdims=True)
        p = np.where(see, np.exp(s - L[:, x][:, None]), 0.0)
        dp = G[:, x] @ V[:, j].T
        d = p * (dp - (G[:, x] * O[:, x]).sum(1, keepdims=True))
        m = p * (np.abs(G[:, x]) @ np.abs(V[:, j]).T + (np.abs(G[:, x]) * np.abs(O[:, x])).sum(1, keepdims=True)) + np.abs(d)
        heads = slice(j * g, (j + 1) * g)
        top = np.linalg.norm(G[:, heads], axis=2).max(1, keepdims=True) * np.linalg.norm(V[:, j], axis=1).max()
        top = top + np.maximum(top, np.abs((G * O).sum(2))[:, heads].max(1, keepdims=True))
        tiny = h * 2.0 ** -38 * see * top
        e = (2 * u + 2 * ds + 2.0 ** -15) * m + tiny
        val["dq"][:, x] = scale * d @ K[:, j]
        err["dq"][:, x] = scale * e @ np.abs(K[:, j])
        e = e + sh * 2.0 ** -11 * m
        val["dk"][:, j] += scale * d.T @ Q[:, x]
        err["dk"][:, j] += scale * (e.T @ np.abs(Q[:, x]) + sh * 2.0 ** -39 * (m.T @ np.linalg.norm(Q[:, x], axis=1))[:, None])
        val["dv"][:, j] += p.T @ G[:, x]
        err["dv"][:, j] += (((u + sh * 2.0 ** -11 + 2 * ds + 2.0 ** -18) * p + h * 2.0 ** -40 * see).T @ np.abs(G[:, x])
                            + sh * 2.0 ** -39 * (p.T @ np.linalg.norm(G[:, x], axis=1))[:, None])
    for n in val:
        err[n] += u * np.abs(val[n]) + h * 2.0 ** -25
    return val, err


@pytest.mark.parametrize("dt", [BF, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hk,D", [(6, 2, 64), (64, 1, 128), (20, 1, 128)])
@pytest.mark.parametrize("K,window,size,nats", [(40, 128, 1, 0), (128, 33, 1, 0), (200, 200, 1, 0), (40, 128, 2 ** 10, 0),
                                                (200, 33, 2 ** 10, 0), (40, 33, 2 ** 13, 12.5), (40, 33, 2 ** 13, 15),
                                                (200, 33, 2 ** 13, 15)])
def test_gradients_of_two_calls_joined_by_lse(K, window, size, nats, Hq, Hk, D, dt):
    """One softmax over selected entries and the last tokens, which are two calls: each call's gradients, from the
    joined out and lse, are its keys' part, whatever the lengths of its list and the weights and sizes of the other's
    values (nats: what the entries' scores are above)."""
    T, W = 230, 300
    q, kt, vt, do = _inputs([T], [T], Hq, Hk, D, dt, seed=38)
    _, ke, ve, _ = _inputs([T], [W], Hq, Hk, D, dt, seed=39)
    vt, do = (vt.float() * size).to(dt), (do.float() / min(size, 16)).to(dt)
    idx = _lists([T], [W], K, 1, seed=19)
    idx[:3] = -1  # rows of no entry
    scale = D ** -0.5
    if nats:
        q[..., 0], ke[..., 0], kt[..., 0] = 4.0, nats / (4 * scale), 0.0
    c = lambda t: t.cuda()  # noqa: E731
    entries = lambda: (c(q), c(ke), c(ve))  # noqa: E731
    ae, aw = (c(idx), c(_cu([T])), c(_cu([W])), scale), (None, c(_cu([T])), c(_cu([T])), scale)
    oe, le = csa.sparse_attn_forward(*entries(), *ae, causal=False)
    ow, lw = csa.sparse_attn_forward(c(q), c(kt), c(vt), *aw, window=window)
    lse = torch.logaddexp(le, lw)
    out = ((le - lse).exp()[..., None] * oe + (lw - lse).exp()[..., None] * ow).to(dt)
    ge = csa.sparse_attn_backward(c(do), *entries(), out, lse, *ae, causal=False)
    gw = csa.sparse_attn_backward(c(do), c(q), c(kt), c(vt), out, lse, *aw, window=window)
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK
    see_e = np.zeros((T, W), dtype=bool)
    r, s = np.nonzero(idx.numpy() >= 0)
    see_e[r, idx.numpy()[r, s]] = True
    at = np.arange(T)
    see_w = (at[None] <= at[:, None]) & (at[None] > at[:, None] - window)
    for name, got, k, v, see in (("entries", ge, ke, ve, see_e), ("window", gw, kt, vt, see_w)):
        val, err = masked(q, k, v, do, out, lse, see, scale, dt)
        for n, t in zip(("dq", "dk", "dv"), got):
            x = np.abs(f64(t) - val[n]) / (err[n] + 1e-30)
            assert x.max() <= 1, (name, n, float(x.max()))


@pytest.mark.parametrize("Hq,Hk,D,dt,K,block", [(65, 1, 128, BF, 20, 2), (134, 2, 64, FP16, 150, 1), (101, 1, 128, FP16, 9, 4),
                                                (254, 2, 64, BF, 70, 4)])
def test_gradients_of_odd_groups_of_more_than_64_heads(Hq, Hk, D, dt, K, block):
    lq, lk = [13, 0, 5], [129, 3, 300]
    q, k, v, do = _inputs(lq, lk, Hq, Hk, D, dt, seed=42)
    _run(q, k, v, do, _lists(lq, lk, K, block, seed=20), _cu(lq), _cu(lk), D ** -0.5, block=block, causal=False)
