"""Scales that attention over listed blocks takes, as the host checks them."""
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


def test_scales_whose_base_2_form_passes_fp32_are_refused(lib):
    fake = ctypes.c_void_p(0x10000)  # never dereferenced: no rows, or refused
    for scale, rows, want in ((2.0 ** 127, 0, abi.CSA_OK), (2.4e38, 10, abi.CSA_ERR_UNSUPPORTED), (3.4e38, 10, abi.CSA_ERR_UNSUPPORTED),
                              (float("inf"), 10, abi.CSA_ERR_INVALID_ARG)):
        p = sparse.SparseProblem(N=1, Tq=rows, Tk=10, Hq=1, Hk=1, D=64, top_k=1, block=1, dtype=abi.CSA_BF16, scale=scale)
        got = lib.csa_sparse_attn_forward(ctypes.byref(p), *[fake] * 6, None, None, fake, fake, fake, 1 << 40, None)
        assert got == want, scale
        if rows:
            assert lib.csa_sparse_attn_backward(ctypes.byref(p), *[fake] * 9, None, *[fake] * 4, 1 << 40, None) == want
            assert lib.csa_sparse_attn_workspace_size(ctypes.byref(p), 1) == 0
