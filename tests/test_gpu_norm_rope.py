"""Norm + rotation of queries and keys on the GPU against the fp64 definition.

Tolerances, from the arithmetic: every output is computed in fp32 and rounded
once, which is off by at most u = eps/2 of the output type, relative.  Before
that a value is a sum of two products of fp32 factors: the norm factor (a sum
of up to 256 squares and rsqrtf: 2^-20), cosine and sine (angle error below
2e-7 < 2^-22, two roundings) and the products: 2^-19 of the magnitudes summed.
The gradients of x add one mean over D: 2^-18 of the magnitudes.  The weights'
gradients add up to a few hundred terms in sequence: 2^-15 of the magnitudes.
"""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu

BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    csa.load()


def _rand(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, dtype=torch.float32).to(dtype)


def _angles(pos, rot, theta):
    return pos.double().numpy()[:, None] * theta ** (-np.arange(0, rot, 2) / rot)[None]


def _close(got, want, mag, rel):
    u = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 2.0 ** -24
    err = np.abs(A.f64(got) - want)
    bound = u * np.abs(want) + rel * mag + 1e-30
    assert np.isfinite(A.f64(got)).all()
    assert (err <= bound * 1.001).all(), float((err / bound).max())


CASES = [  # T, Hq, Hk, D, rot, off, interleaved, dtype, wdtype, first position
    (1, 1, 1, 8, 8, 0, True, BF, BF, 0),
    (1, 64, 8, 128, 128, 0, False, BF, BF, 131071),
    (7, 3, 1, 128, 64, 64, True, FP16, F32, 5),
    (33, 5, 5, 64, 64, 0, False, FP16, FP16, 1000),
    (130, 12, 3, 32, 16, 16, True, F32, F32, 900001),
    (65, 4, 2, 96, 32, 8, False, BF, F32, -70),
    (19, 2, 1, 256, 256, 0, False, F32, BF, 77),
    (257, 1, 0, 40, 32, 8, False, BF, BF, 3),
    (301, 9, 1, 248, 240, 8, False, FP16, F32, 12345),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradients(case):
    T, Hq, Hk, D, rot, off, inter, dt, wt, p0 = case
    gen = torch.Generator().manual_seed(T * 31 + D)
    # views into a wider row, as a projection leaves them
    wide = _rand(gen, T, Hq + Hk + 1, D + 8, dtype=dt)
    wide[:, :, D:] = float("nan")  # what stands between the rows is not read
    q, k = wide[:, :Hq, :D], (wide[:, Hq:Hq + Hk, :D] if Hk else None)
    qw = (1 + 0.3 * _rand(gen, D, dtype=F32)).to(wt)
    kw = (1 + 0.3 * _rand(gen, D, dtype=F32)).to(wt) if Hk else None
    gq, gk = _rand(gen, T, Hq, D, dtype=dt), (_rand(gen, T, Hk, D, dtype=dt) if Hk else None)
    pos = torch.arange(T) + p0
    fr = csa.rope_freqs(rot, 50000.0)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    wide_g = wide.cuda()
    qg, kg = wide_g[:, :Hq, :D], (wide_g[:, Hq:Hq + Hk, :D] if Hk else None)
    arg = dict(eps=1e-5, rot_offset=off, interleaved=inter)
    yq, yk = csa.norm_rope(qg, kg, c(qw), c(kw), pos.cuda(), fr, **arg)
    dq, dk, dqw, dkw = csa.norm_rope_backward(c(gq), c(gk), qg, kg, c(qw), c(kw), pos.cuda(), fr, **arg)
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK
    ang = _angles(pos, rot, 50000.0)
    for x, w, g, y, dx, dw in ((q, qw, gq, yq, dq, dqw), (k, kw, gk, yk, dk, dkw)):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        X, W, G = A.f64(x), A.f64(w), A.f64(g)
        ref, mag = A.norm_rope(X, W, ang, 1e-5, off, inter)
        _close(y, ref, mag, 2.0 ** -19)
        rx, mx, rw, mw = A.norm_rope_vjp(G, X, W, ang, 1e-5, off, inter)
        _close(dx, rx, mx, 2.0 ** -18)
        _close(dw, rw, mw, 2.0 ** -15)


# More rows than one round over the GPU holds, the last one short, tokens across units: every group of lanes
# goes on to further rows.
ROUNDS = [
    (1601, 45, 7, 128, 64, 64, True, BF, BF, 11),
    (3001, 13, 1, 256, 256, 0, False, FP16, F32, 0),
    (20011, 3, 2, 128, 128, 0, False, F32, F32, 900001),
    (300007, 1, 1, 32, 32, 0, False, BF, BF, 5),
]


@pytest.mark.parametrize("case", ROUNDS, ids=str)
def test_several_rounds(case):
    test_forward_and_gradients(case)


def test_gradient_by_differences():
    # directional difference of sum(y * g) in fp32 against <dx, d> + <dw, e>
    gen = torch.Generator().manual_seed(3)
    T, H, D = 6, 2, 64
    x, w, g = _rand(gen, T, H, D, dtype=F32), 1 + 0.2 * _rand(gen, D, dtype=F32), _rand(gen, T, H, D, dtype=F32)
    d, e = _rand(gen, T, H, D, dtype=F32), _rand(gen, D, dtype=F32)
    pos, fr = torch.arange(T).cuda() * 100, csa.rope_freqs(64)
    h = 2.0 ** -8

    def value(s):
        y, _ = csa.norm_rope((x + s * h * d).cuda(), None, (w + s * h * e).cuda(), None, pos, fr)
        return float((y.double().cpu() * g.double()).sum())

    dx, _, dw, _ = csa.norm_rope_backward(g.cuda(), None, x.cuda(), None, w.cuda(), None, pos, fr)
    want = float((dx.double().cpu() * d.double()).sum() + (dw.double().cpu() * e.double()).sum())
    # third derivatives: order h^2 of the sum's magnitude; fp32 values: 2^-19 / h
    size = float((g.abs() * (d.abs() + e.abs())).double().sum()) * 4
    assert abs((value(1) - value(-1)) / (2 * h) - want) <= size * (h * h + 2.0 ** -19 / h)


def test_positions_wrap_exactly():
    # a table of exact fractions of a turn: a quarter per position, and 2^-40: any 64-bit position is exact
    fr = torch.tensor([1 << 62, 1 << 24, 0, 1 << 63 - 1], dtype=torch.int64).cuda()
    x = torch.randn(4, 1, 8, generator=torch.Generator().manual_seed(0)).cuda()
    pos = torch.tensor([0, (1 << 40) + 1, -(1 << 40) - 1, (1 << 62) + 3], dtype=torch.int64)
    y, _ = csa.norm_rope(x, None, torch.ones(8).cuda(), None, pos.cuda(), fr, eps=0.0, interleaved=True)
    turns = [[(int(p) * f) % (1 << 64) / 2.0 ** 64 for f in (1 << 62, 1 << 24, 0, 1 << 62)] for p in pos]
    ref, mag = A.norm_rope(A.f64(x), np.ones(8), 2 * np.pi * np.array(turns), 0.0, 0, True)
    _close(y, ref, mag, 2.0 ** -19)


def test_no_tokens():
    fr = csa.rope_freqs(32)
    e = lambda h: torch.empty(0, h, 32, dtype=BF, device="cuda")  # noqa: E731
    w = torch.ones(32, dtype=BF, device="cuda")
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    yq, yk = csa.norm_rope(e(4), e(2), w, w, pos, fr)
    assert yq.shape == (0, 4, 32) and yk.shape == (0, 2, 32)
    _, _, dqw, dkw = csa.norm_rope_backward(e(4), e(2), e(4), e(2), w, w, pos, fr)
    assert not dqw.any() and not dkw.any()


def test_weight_gradients_repeat_bit_for_bit():
    gen = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn(3000, 8, 128, generator=gen, device="cuda", dtype=BF)
    w, pos, fr = torch.ones(128, device="cuda"), torch.arange(3000, device="cuda"), csa.rope_freqs(128)
    one = csa.norm_rope_backward(q, q, q, q, w, w, pos, fr)
    two = csa.norm_rope_backward(q, q, q, q, w, w, pos, fr)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    assert torch.equal(one[0], one[1])


def test_side_stream_and_graph():
    gen = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(50, 4, 64, generator=gen, device="cuda", dtype=BF)
    w, pos, fr = torch.ones(64, device="cuda", dtype=BF), torch.arange(50, device="cuda"), csa.rope_freqs(64)
    ref, _ = csa.norm_rope(q, None, w, None, pos, fr)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, _ = csa.norm_rope(q, None, w, None, pos, fr, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap, _ = csa.norm_rope(q, None, w, None, pos, fr)
    q.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, -ref)


def test_binding_refuses():
    q = torch.zeros(3, 4, 64, dtype=BF, device="cuda")
    w, pos, fr = torch.ones(64, dtype=BF, device="cuda"), torch.arange(3, device="cuda"), csa.rope_freqs(64)
    for kw in (dict(pos=pos.int()), dict(pos=pos[:2]), dict(w=w[:32]), dict(q=q.transpose(1, 2)), dict(q=q.double()),
               dict(q=q[:1].expand(3, 4, 64))):
        a = dict(q=q, w=w, pos=pos)
        a.update(kw)
        with pytest.raises((ValueError, csa.CsaError)):
            csa.norm_rope(a["q"], None, a["w"], None, a["pos"], fr)
    with pytest.raises(csa.CsaError):  # a base off the 16-byte grid
        csa.norm_rope(torch.zeros(3, 4, 72, dtype=BF, device="cuda")[..., 4:68], None, w, None, pos, fr)
