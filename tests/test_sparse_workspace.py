"""Workspaces of the gradients of attention over listed blocks, as the host computes them."""
import ctypes
import os

import pytest

from sparse_attention_indexer_csa_gb300 import abi, sparse


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from sparse_attention_indexer_csa_gb300 import build
        build.build()
    return sparse.load()


def _bytes(lib, heads, rows=1000):
    p = sparse.SparseProblem(N=1, Tq=rows, Tk=4096, Hq=heads, Hk=1, D=128, top_k=256, block=1, dtype=abi.CSA_BF16, scale=0.1)
    return int(lib.csa_sparse_attn_workspace_size(ctypes.byref(p), 1))


def test_groups_of_any_size_take_the_shares_of_one_or_two_items(lib):
    one, two = _bytes(lib, 64), _bytes(lib, 128)
    # a share of dk and of dv, 2 bytes a value, and its powers of two
    assert two - one >= 1000 * 256 * (2 * 128 * 2 + 2)
    for heads in range(1, 65):
        assert _bytes(lib, heads) <= one
    for heads in range(65, 129):
        assert one < _bytes(lib, heads) <= two
