"""Pins of oracle/attn_oracle.py (no GPU): hand values, differences, invariants."""
import math

import numpy as np
import pytest

from oracle import attn_oracle as A


def test_norm_rope_by_hand():
    # x = (3, 4): mean square 12.5; a quarter turn sends (u, v) to (-v, u)
    x = np.array([[[3.0, 4.0]]])
    r = 1 / math.sqrt(12.5)
    y, _ = A.norm_rope(x, np.array([1.0, 2.0]), np.array([[math.pi / 2]]), 0.0, 0, True)
    assert np.allclose(y, [[[-8 * r, 3 * r]]])


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_gradient_by_differences(inter):
    rng = np.random.default_rng(0)
    x, w, dy = rng.standard_normal((3, 2, 16)), 1 + 0.3 * rng.standard_normal(16), rng.standard_normal((3, 2, 16))
    ang = rng.standard_normal((3, 4)) * 5
    f = lambda x, w: (A.norm_rope(x, w, ang, 1e-3, 8, inter)[0] * dy).sum()  # noqa: E731
    dx, _, dw, _ = A.norm_rope_vjp(dy, x, w, ang, 1e-3, 8, inter)
    h = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(16):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * h) - dw[i]) < 1e-7


def test_attention_by_hand():
    # two keys of equal score, then a row that sees one key and a row that sees none
    k = np.array([[[1.0, 0.0]], [[1.0, 0.0]]])
    v = np.array([[[2.0, 0.0]], [[4.0, 6.0]]])
    q = np.ones((3, 1, 2))
    r = A.attention(q, k, v, [0, 3], [0, 2], 0.5)
    assert np.allclose(r["out"][:, 0], [[0, 0], [2, 0], [3, 3]])
    assert r["lse"][0, 0] == -np.inf and np.allclose(r["lse"][1:, 0], [0.5, 0.5 + math.log(2)])


def test_attention_gradient_by_differences():
    rng = np.random.default_rng(1)
    cu_q, cu_k = [0, 3, 3, 7], [0, 5, 6, 8]
    q, k, v, g = (rng.standard_normal(s) for s in ((7, 4, 3), (8, 2, 3), (8, 2, 3), (7, 4, 3)))
    f = lambda q, k, v: (A.attention(q, k, v, cu_q, cu_k, 0.7)["out"] * g).sum()  # noqa: E731
    r = A.attention(q, k, v, cu_q, cu_k, 0.7, dout=g)
    h = 1e-6
    args = [q, k, v]
    for n, name in enumerate(("dq", "dk", "dv")):
        for i in np.ndindex(args[n].shape):
            d = np.zeros_like(args[n])
            d[i] = h
            hi, lo = list(args), list(args)
            hi[n], lo[n] = args[n] + d, args[n] - d
            assert abs((f(*hi) - f(*lo)) / (2 * h) - r[name][i]) < 1e-7


def test_attention_of_packed_sequences_is_that_of_each():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal(s) for s in ((9, 2, 4), (11, 1, 4), (11, 1, 4)))
    whole = A.attention(q, k, v, [0, 4, 9], [0, 6, 11], 0.5, k_len=[5, 5])
    one = A.attention(q[4:], k[6:], v[6:], [0, 5], [0, 5], 0.5)
    two = A.attention(q[:4], k[:5], v[:5], [0, 4], [0, 5], 0.5)
    assert np.array_equal(whole["out"][4:], one["out"]) and np.array_equal(whole["out"][:4], two["out"])
