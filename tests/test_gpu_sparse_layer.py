"""The indexer's selection, attention over it, its gradients and the paged cache together, as examples/sparse_layer.py
runs them.

* The step over the pages against the definition on what the cache holds, with the bounds of test_gpu_sparse.
* The cached keys and values against the prompt's: the same kernel's on the same hidden states but for the projection, a
  library product that may sum in another order for a chunk and so round to a neighbour, 2u of a value (u = 2^-8); a
  key's value is made of two of them (the rotation) and rounded once on each side: 2 * 2u + 2u of the row's largest.
* Selected entries are complete and of the row's document, distinct, in ascending order.
* Weights' gradients against differences of the layer's loss in 64 bits for the selection that the layer made, along the
  gradient itself: see test_gpu_layer for the ten roundings, 10 u of the sum.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from oracle import sparse_oracle as S
from oracle.attn_oracle import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_layer.py")
    spec = importlib.util.spec_from_file_location("sparse_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


LENGTHS = [(300, 9, 129, 514), (5, 128, 4), (1,), (64, 64, 2, 1, 250)]


def _cached(r, i, n):
    """The first n keys and values of document i, by the page table."""
    c = r["cache"]
    page = c.k.shape[1]
    rows = torch.tensor([int(c.table[i, j // page]) * page + j % page for j in range(n)], device="cuda")
    return tuple(f64(t.view(-1, *t.shape[2:])[rows]) for t in (c.k, c.v))


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_a_step_over_the_pages(layer, lengths):
    r = layer.run(lengths)
    kv = [_cached(r, i, n) for i, n in enumerate(lengths)]
    k, v = (np.concatenate([x[i] for x in kv]) for i in range(2))
    u = 2.0 ** -8
    for got, want in ((k, f64(r["k"])), (v, f64(r["v"]))):
        assert (np.abs(got - want) <= 6 * u * np.abs(want).max(-1, keepdims=True)).all()
    n = len(lengths)
    cu_q, cu_k = np.arange(n + 1), np.concatenate([[0], np.cumsum(lengths)])
    ref = S.attention(f64(r["step_q"]), k, v, r["step_idx"].cpu().numpy(), cu_q, cu_k, layer.SCALE, layer.RATE,
                      layer.WINDOW)
    ds = 2.0 ** -16 * ref["smax"][..., None]
    bound = u * np.abs(ref["out"]) + (u + 2 * ds + 2.0 ** -18) * ref["mag_out"]
    assert (np.abs(f64(r["step"]) - ref["out"]) <= bound).all()
    # pages that no token reached are as they were
    used = sum(lengths)
    assert int((~torch.isnan(r["cache"].k[..., 0, 0])).sum()) == used
    assert r["cache"].lens.tolist() == list(lengths)


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_selection(layer, lengths):
    r = layer.run(lengths)
    idx = r["idx"].cpu().numpy()
    pos = r["positions"].cpu().numpy()
    rows, at = np.nonzero(idx >= 0)
    assert ((idx[rows, at] + 1) * layer.RATE <= pos[rows] + 1).all()
    assert ((idx >= 0).sum(1) == np.minimum((pos + 1) // layer.RATE, layer.TOP_K)).all()
    both = (idx[:, 1:] >= 0) & (idx[:, :-1] >= 0)
    assert (np.diff(idx, axis=1)[both] > 0).all()


def _loss64(layer, r, qkv, q_norm, k_norm):
    x, cu = f64(r["x"]), r["cu"].cpu().numpy()
    y = (x @ qkv).reshape(x.shape[0], -1, layer.D)
    q0, k0, v = y[:, :layer.HQ], y[:, layer.HQ:layer.HQ + layer.HK], y[:, layer.HQ + layer.HK:]
    pos, rot = r["positions"].cpu().numpy(), layer.ROT
    ang = pos[:, None] * layer.THETA ** (-2.0 * np.arange(rot // 2) / rot)[None]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]

    def turn(x, w):
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + layer.EPS) * w
        a, b = n[..., layer.D - rot:layer.D - rot // 2], n[..., layer.D - rot // 2:]
        return np.concatenate([n[..., :layer.D - rot], a * c - b * s, a * s + b * c], -1)

    ref = S.attention(turn(q0, q_norm), turn(k0, k_norm), v, r["idx"].cpu().numpy(), cu, cu, layer.SCALE, layer.RATE,
                      layer.WINDOW)
    return 0.5 * ((ref["out"] - r["target"].double().cpu().numpy()) ** 2).mean()


@pytest.mark.parametrize("which", ["qkv", "q_norm", "k_norm"])
def test_gradients_against_differences(layer, which):
    r = layer.run((40, 1, 150), seed=5)
    g = f64(r["grads"][which]) / 2 ** 16
    w = {n: f64(r["weights"][n]) for n in ("qkv", "q_norm", "k_norm")}
    size = np.linalg.norm(g)
    h = 1e-4 * np.linalg.norm(w[which]) / size
    up, down = (_loss64(layer, r, **{**w, which: w[which] + d * h * g}) for d in (1, -1))
    got = (up - down) / (2 * h)
    assert abs(got - size ** 2) <= 10 * 2.0 ** -8 * size ** 2


def test_the_selection_feeds_attention_over_entries():
    """index_fused's [B,S,top_k] read as [B*S,top_k] lists the entries themselves: attention over compressed keys."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    B, T, W, K, D = 2, 200, 50, 12, 128
    idx = csa.index_fused(r(B, 64, T, D), r(B, W, D), r(B, T, 64), 0.1, 4, K)
    q, k, v = r(B * T, 8, D), r(B * W, 1, D), r(B * W, 1, D)
    cu = lambda n: torch.arange(B + 1, device="cuda", dtype=torch.int32) * n  # noqa: E731
    out, lse = csa.sparse_attn_forward(q, k, v, idx.view(B * T, K), cu(T), cu(W), 0.1, causal=False)
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK
    rows = csa.index_gather(k.view(B, W, D), idx).double().cpu()  # [B,T,K,D], zeros for -1
    vals = csa.index_gather(v.view(B, W, D), idx).double().cpu()
    s = torch.einsum("bthd,btkd->bthk", q.view(B, T, 8, D).double().cpu(), rows) * 0.1
    s = s.masked_fill((idx.cpu() < 0)[:, :, None], -float("inf"))
    some = (idx.cpu() >= 0).any(-1)
    p = torch.softmax(s[some], -1)
    want = torch.einsum("nhk,nkd->nhd", p, vals[some])
    got = out.view(B, T, 8, D).double().cpu()
    mag = torch.einsum("nhk,nkd->nhd", p, vals[some].abs())
    # u of the output, u of p, and 2^-12 for the scores' fp32 sums (|q||k| scale below 2^4)
    assert ((got[some] - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11) * mag).all()
    assert not got[~some].any() and (~some).sum() == 2 * 3
