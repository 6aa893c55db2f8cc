"""Pins of oracle/sparse_oracle.py (no GPU): hand values, the dense definition, differences."""
import numpy as np
import pytest

from oracle import attn_oracle as A
from oracle import sparse_oracle as S


def test_counts_by_hand():
    # blocks of 2 over 7 keys, window 2: positions 6 and 3
    n = S.counts([[0, 3, -1], [1, 0, 0]], [6, 3], 7, 2, 2, True)
    assert n.tolist() == [[1, 1, 0, 0, 0, 1, 1], [2, 2, 1, 1, 0, 0, 0]]
    # block 3 holds key 6 alone, which lies in the window; key 5 is in it unlisted
    n = S.counts([[3, -1, 1]], [6], 7, 2, 0, False)
    assert n.tolist() == [[0, 0, 1, 1, 0, 0, 1]]
    assert S.counts([[0]], [-1], 3, 1, 2, True).tolist() == [[0, 0, 0]]


def _random(seed, lq, lk, Hq=4, Hk=2, D=8):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s)  # noqa: E731
    return r(sum(lq), Hq, D), r(sum(lk), Hk, D), r(sum(lk), Hk, D), r(sum(lq), Hq, D)


@pytest.mark.parametrize("block,window", [(1, 0), (2, 3), (4, 100)])
def test_all_blocks_listed_is_dense_attention(block, window):
    lq, lk = [5, 0, 7], [9, 2, 4]
    q, k, v, do = _random(1, lq, lk)
    cu_q, cu_k = np.cumsum([0, *lq]), np.cumsum([0, *lk])
    idx = np.tile(np.arange(max(lk)), (sum(lq), 1))
    idx = np.where(idx * block < np.repeat(lk, lq)[:, None], idx, -1)
    got = S.attention(q, k, v, idx, cu_q, cu_k, 0.3, block, window, True, None, do)
    want = A.attention(q, k, v, cu_q, cu_k, 0.3, True, None, do)
    for n in ("out", "lse", "dq", "dk", "dv"):
        assert np.allclose(got[n], want[n], atol=1e-12), n


def test_gradients_by_differences_with_a_block_listed_twice():
    lq, lk = [3, 2], [6, 5]
    q, k, v, do = _random(2, lq, lk)
    cu_q, cu_k = np.cumsum([0, *lq]), np.cumsum([0, *lk])
    idx = np.array([[0, 0], [1, 0], [-1, 1], [0, 1], [1, 1]])
    f = lambda q, k, v: (S.attention(q, k, v, idx, cu_q, cu_k, 0.5, 2, 1)["out"] * do).sum()  # noqa: E731
    res = S.attention(q, k, v, idx, cu_q, cu_k, 0.5, 2, 1, dout=do)
    rng = np.random.default_rng(3)
    for n, x in (("dq", 0), ("dk", 1), ("dv", 2)):
        d = [np.zeros_like(t) for t in (q, k, v)]
        d[x] = rng.standard_normal(d[x].shape)
        up = f(*(t + 1e-6 * e for t, e in zip((q, k, v), d)))
        down = f(*(t - 1e-6 * e for t, e in zip((q, k, v), d)))
        assert abs((up - down) / 2e-6 - (res[n] * d[x]).sum()) < 1e-7
