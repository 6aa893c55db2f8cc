"""Append to a paged cache where the table ends before the tokens do."""
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from test_gpu_append import BF, _call, _case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    csa.load()


def test_tokens_past_a_narrow_table_are_reported_and_not_stored():
    """The table is a view of a wider one, whose next column names a page of the pool: the tokens past the width have no
    other cause to be refused."""
    s, rows = _case([6, 5], [20, 27], 8, 4, 2, 64, BF, BF, seed=6)
    fr = csa.rope_freqs(64)
    full = dict(s, k_pages=s["k_pages"].clone(), v_pages=s["v_pages"].clone())
    want_q = _call(full, fr)
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK
    wide = s["table"].clone()
    wide[1, 4] = wide[0, 0]
    s["k_len"][1] = 8 * 4 + 5  # the five tokens stand at places 32 to 36, in page 4 of four
    want_k, want_v = s["k_pages"].clone(), s["v_pages"].clone()
    for w, x in ((want_k, full["k_pages"]), (want_v, full["v_pages"])):
        w.view(-1, 2, 64)[rows[:6]] = x.view(-1, 2, 64)[rows[:6]]
    got = _call(dict(s, table=wide[:, :4]), fr)
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_ERR_DEVICE
    assert torch.equal(got, want_q)
    assert torch.equal(s["k_pages"], want_k) and torch.equal(s["v_pages"], want_v)
