"""GB300 (sm_103a) CSA indexer: per-row top-k selection of compressed KV
entries by the head-reduced score  sum_h w[b,s,h] * ReLU(scale * q.k), and the
operators around it: norm and rotation of queries and keys, attention of packed
sequences, with their gradients.

The compute lives in ``libcsa_index.so`` (hand-written CUDA behind the C ABIs
of ``include/csa_index.h`` and ``include/csa_attn.h``); this package is its
build script and a thin ctypes binding.
"""
from .abi import (CSA_BF16, CSA_ERR_CUDA, CSA_Q_HEAD_MAJOR, CSA_Q_SEQ_MAJOR, CSA_ERR_DEVICE, CSA_ERR_INVALID_ARG,  # noqa: F401
                  CSA_ERR_TIMEOUT, CSA_ERR_UNSUPPORTED, CSA_F32, CSA_OK, CsaError, Problem,
                  device_status, fused_host_bytes, index_backward, index_decode, index_gather, index_fused,
                  index_fused_host, index_fused_host_raw, index_fused_raw, index_score,
                  index_score_raw, index_topk, index_topk_raw, load, make_problem,
                  selftest_timeout, workspace_size)
from .attn import (CSA_F16, AttnProblem, NormRopeProblem, attn_backward, attn_forward,  # noqa: F401
                   attn_workspace_size, make_attn_problem, make_norm_rope_problem, norm_rope, norm_rope_backward,
                   rope_freqs)
