"""The operators together, as examples/packed_layer.py runs them.

* A token computed as a step over the cache against the same row of the prompt.  Both
  are within (2u + 2 ds + 2^-18) max|v| of the exact row, u = 2^-8 (bf16; P is rounded, then
  the output) and ds = 2^-16 scale |q||k|; the query and key are the same kernel's
  on the same values, but for the projection, a library product that may sum in another
  order and so round to a neighbour: one more 2u of the value, and 2u of q and k each,
  which move a score by at most 4u scale |q||k|.
* Selected entries belong to the row's document and its past.
* Weights' gradients against differences of the layer's loss in 64 bits, along the
  gradient itself: with g the computed gradient and h a step, (L(w + h g) - L(w - h g)) / 2h = |g|^2
  up to the roundings: dout, P, dS, the outputs of each backward and of the product are
  rounded to 8 bits; those of the forward (q, k, out) shift where the gradient is taken.
  Ten roundings of at most u each, all with the sign that hurts: 10 u = 2^-4.6 of the sum.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "packed_layer.py")
    spec = importlib.util.spec_from_file_location("packed_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


LENGTHS = [(300, 1, 129, 514), (5, 128, 3), (1,), (64, 64, 2, 1, 250)]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_a_step_gives_the_prompts_row(layer, lengths):
    r = layer.run(lengths)
    u = 2.0 ** -8
    q, k = (A.f64(r[n]) for n in ("q", "k"))
    s = layer.SCALE * np.linalg.norm(q, axis=-1).max() * np.linalg.norm(k, axis=-1).max()
    bound = (2 * (2 * u + 2 * 2.0 ** -16 * s + 2.0 ** -18) + 2 * u + 2 * 4 * u * s) * np.abs(A.f64(r["v"])).max()
    got, want = A.f64(r["step"]), A.f64(r["out"][r["last"]])
    assert np.isfinite(got).all() and np.abs(got - want).max() <= bound
    # nearly all rows have the very same projections: their bound has no term of the scores
    tight = (2 * (2 * u + 2 * 2.0 ** -16 * s + 2.0 ** -18) + 2 * u) * np.abs(A.f64(r["v"])).max()
    assert np.median(np.abs(got - want)) <= tight


@pytest.mark.parametrize("lengths", LENGTHS[:2], ids=str)
def test_selection_stays_in_the_document(layer, lengths):
    r = layer.run(lengths)
    idx = r["idx"][0].cpu().numpy()
    doc = np.repeat(np.arange(len(lengths)), lengths)
    rows, at = np.nonzero(idx >= 0)
    entry = idx[rows, at]
    assert (doc[entry * layer.RATE] == doc[rows]).all() and ((entry + 1) * layer.RATE <= rows + 1).all()


def _loss64(layer, r, qkv, q_norm, k_norm, target):
    x, w, cu = A.f64(r["x"]), r["weights"], r["cu"].cpu().numpy()
    y = (x @ qkv).reshape(x.shape[0], -1, layer.D)
    q0, k0, v = y[:, :layer.HQ], y[:, layer.HQ:layer.HQ + layer.HK], y[:, layer.HQ + layer.HK:]
    pos, rot = r["positions"].cpu().numpy(), layer.ROT
    ang = pos[:, None] * layer.THETA ** (-2.0 * np.arange(rot // 2) / rot)[None]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]

    def turn(x, w):
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + layer.EPS) * w
        a, b = n[..., layer.D - rot:layer.D - rot // 2], n[..., layer.D - rot // 2:]
        return np.concatenate([n[..., :layer.D - rot], a * c - b * s, a * s + b * c], -1)

    ref = A.attention(turn(q0, q_norm), turn(k0, k_norm), v, cu, cu, layer.SCALE)
    return 0.5 * ((ref["out"] - target) ** 2).mean()


@pytest.mark.parametrize("which", ["qkv", "q_norm", "k_norm"])
def test_gradients_against_differences(layer, which):
    lengths = (40, 1, 150)
    r = layer.run(lengths, seed=5)
    gen = torch.Generator().manual_seed(6)  # as run(): the hidden states, then the target
    torch.randn(sum(lengths), layer.WIDTH, generator=gen)
    target = torch.randn(r["out"].shape, generator=gen).double().numpy()
    g = A.f64(r["grads"][which]) / 2 ** 16
    w = {n: A.f64(r["weights"][n]) for n in ("qkv", "q_norm", "k_norm")}
    size = np.linalg.norm(g)
    h = 1e-4 * np.linalg.norm(w[which]) / size
    up, down = (_loss64(layer, r, **{**w, which: w[which] + d * h * g}, target=target) for d in (1, -1))
    got = (up - down) / (2 * h)
    assert abs(got - size ** 2) <= 10 * 2.0 ** -8 * size ** 2
