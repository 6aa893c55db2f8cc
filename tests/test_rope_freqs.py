"""The table of csa_rope_freqs against decimal arithmetic of 60 digits (no GPU)."""
import decimal
import math
import os

import numpy as np
import pytest

import sparse_attention_indexer_csa_gb300 as csa
from sparse_attention_indexer_csa_gb300 import abi

D = decimal.Decimal
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(abi.LIB_PATH):
        from sparse_attention_indexer_csa_gb300 import build
        build.build()


@pytest.mark.parametrize("theta,rot", [(10000.0, 64), (10000.0, 128), (500000.0, 256), (1.5, 2), (1e18, 48),
                                       (1.0 + 2.0 ** -40, 16), (math.pi * 1e6, 8)])
def test_all_64_bits_of_the_fraction(theta, rot):
    """At position p an error of the table is p times as large, so every bit counts.  Half a unit of the last
    place for the rounding, and a little for the arithmetic before it."""
    with decimal.localcontext() as c:
        c.prec = 60
        t = csa.rope_freqs(rot, theta, device="cpu").numpy().view(np.uint64)
        for i, f in enumerate(t):
            want = (D(theta).ln() * (-2 * i) / rot).exp() / (2 * PI) * 2 ** 64
            assert abs(D(int(f)) - want) <= D("0.51"), i


@pytest.mark.gpu
@pytest.mark.parametrize("first", [10 ** 12, -(10 ** 12) - 7, 3 * 10 ** 9])
def test_far_positions_on_the_gpu(first):
    """Rotation at positions around 1e12 in fp32.  The table's half units are 2.7e-8 of a turn there, 1.7e-7
    radians; cosine, sine, norm and products as at any position (2^-19 of the magnitudes, the angle's 2e-7 in it)."""
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from oracle import attn_oracle as A

    theta, rot = 10000.0, 64
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(9, 2, rot, generator=gen)
    pos = first + torch.arange(9) * 1001
    y, _ = csa.norm_rope(x.cuda(), None, torch.ones(rot).cuda(), None, pos.cuda(), csa.rope_freqs(rot, theta))
    with decimal.localcontext() as c:
        c.prec = 60
        f = [(D(theta).ln() * (-2 * i) / rot).exp() for i in range(rot // 2)]
        ang = np.array([[float((int(p) * w) % (2 * PI)) for w in f] for p in pos])
    want, mag = A.norm_rope(A.f64(x), np.ones(rot), ang, 1e-6, 0, False)
    assert (np.abs(A.f64(y) - want) <= 2.0 ** -24 * np.abs(want) + (2.0 ** -19 + 1.8e-7) * mag).all()
