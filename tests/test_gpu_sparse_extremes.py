"""Gradients of attention over listed blocks where scales, magnitudes or hidden values are extreme.

Tolerances are those of test_gpu_sparse (its docstring derives them); they scale with the inputs.
"""
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
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
