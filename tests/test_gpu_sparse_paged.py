"""Attention over listed blocks of a paged cache, on the paths that no window takes: bit for bit as over packed keys, which
test_gpu_sparse holds against the definition."""
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from test_gpu_sparse import BF, FP16, _cu, _inputs, _lists, _paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    csa.load()


@pytest.mark.parametrize("block,page", [(4, 4), (4, 24), (8, 64), (64, 16), (128, 100)])
@pytest.mark.parametrize("causal", [True, False])
def test_paged_blocks_without_a_window_give_the_packed_bits(causal, block, page):
    """Four keys a lane (blocks and pages of multiples of four), and copies of few, some and many query heads."""
    lq, lk = [3, 1, 0, 2], [700, 129, 5, 2]
    for Hq, Hk, D, dt in ((8, 2, 128, BF), (40, 1, 64, FP16), (100, 1, 128, BF), (18, 2, 64, BF)):
        q, k, v, _ = _inputs(lq, lk, Hq, Hk, D, dt, seed=page)
        idx = _lists(lq, lk, 20, block, seed=page)
        kp, vp, table = _paged(k, v, lk, page)
        c = lambda t: t.cuda()  # noqa: E731
        kw = dict(block=block, causal=causal)
        want = csa.sparse_attn_forward(c(q), c(k), c(v), c(idx), c(_cu(lq)), c(_cu(lk)), 0.1, **kw)
        got = csa.sparse_attn_paged(c(q), c(kp), c(vp), c(table), c(idx), c(_cu(lq)),
                                    torch.tensor(lk, dtype=torch.int32).cuda(), 0.1, **kw)
        torch.cuda.synchronize()
        assert csa.device_status() == csa.CSA_OK
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and want[0].any()


def test_entries_of_a_paged_cache_one_token_of_many_sequences():
    """The decode step over compressed entries: lists without a causal border, more sequences than the lanes hold."""
    N, lk = 40, [(7 * i) % 90 for i in range(40)]
    q, k, v, _ = _inputs([1] * N, lk, 64, 1, 128, BF, seed=50)
    idx = _lists([1] * N, lk, 30, 1, seed=21)
    kp, vp, table = _paged(k, v, lk, 16)
    c = lambda t: t.cuda()  # noqa: E731
    want = csa.sparse_attn_forward(c(q), c(k), c(v), c(idx), c(_cu([1] * N)), c(_cu(lk)), 0.1, causal=False)
    got = csa.sparse_attn_paged(c(q), c(kp), c(vp), c(table), c(idx), c(_cu([1] * N)),
                                torch.tensor(lk, dtype=torch.int32).cuda(), 0.1, causal=False)
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert not got[0][0].any() and (got[1][0] == -float("inf")).all()  # a sequence without keys
