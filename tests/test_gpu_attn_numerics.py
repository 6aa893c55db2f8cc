"""Attention on the GPU where lengths, magnitudes or infinities are extreme.

Each tolerance counts the roundings named beside it; u = eps/2 of the storage
type, and ds = 2^-16 of the largest scale*|q|.|k| bounds a score's error (fp32
sums of exact products).
"""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu

BF, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    csa.load()


def _cu(*lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def _ok():
    torch.cuda.synchronize()
    assert csa.device_status() == csa.CSA_OK


def test_gradients_of_keys_far_before_the_rows():
    """One row of 128 heads over 17 million keys: the distance of an early key from the row, times
    the heads, passes 2^31.

    All keys and values are zero but for a few, so that the definition is a sum over those and one more term of
    weight n0.  The forward's out and lse are the definition's, rounded.  dk and dv: the roundings of p or of ds
    (u), the score's error (2 ds), delta from the rounded out (u sum |dout||out|), fp32 sums of 64
    products (2^-15), the output's own (u).
    """
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB of device memory")
    lk, H, D, scale = 17_000_000, 128, 64, 0.125
    gen = torch.Generator().manual_seed(41)
    r = lambda *s: torch.randn(*s, generator=gen).to(BF)  # noqa: E731
    at = [0, 5, 200, lk // 2, lk - 1]
    n0 = lk - len(at)
    q, do, kt, vt = r(1, H, D), r(1, H, D), r(len(at), D), r(len(at), D)
    q[..., 0], kt[3, 0] = 4.0, 32.0  # one key weighs as much as all the zero ones
    Q, G, K, V = A.f64(q)[0], A.f64(do)[0], A.f64(kt), A.f64(vt)
    s = scale * Q @ K.T
    z = np.exp(s).sum(1) + n0
    p, p0 = np.exp(s) / z[:, None], 1 / z
    out = torch.from_numpy(p @ V).to(BF)
    O = A.f64(out)
    k, v = (torch.zeros(lk, 1, D, dtype=BF, device="cuda") for _ in range(2))
    k[at, 0], v[at, 0] = kt.cuda(), vt.cuda()
    dq, dk, dv = csa.attn_backward(do.cuda(), q.cuda(), k, v, out[None].cuda(),
                                   torch.from_numpy(np.log(z)).float()[None].cuda(), _cu(1), _cu(lk), scale)
    _ok()
    u = 2.0 ** -8
    ds = 2.0 ** -16 * scale * (np.abs(Q) @ np.abs(K).T).max()
    delta = (G * (p @ V)).sum(1)
    err = u * (np.abs(G) * np.abs(O)).sum(1)  # of delta
    def grads(p, dp, dpm):  # of one key, from its weight in each head, dP and the magnitudes of dP's sum
        d = p * (dp - delta)
        dm = np.abs(d) * (u + 2 * ds) + p * (err + 2.0 ** -15 * dpm)
        gk, gv = scale * d @ Q, p @ G
        return (gk, u * np.abs(gk) + scale * dm @ np.abs(Q) + 2.0 ** -15 * np.abs(scale * d) @ np.abs(Q),
                gv, u * np.abs(gv) + (u + 2 * ds + 2.0 ** -15) * p @ np.abs(G))
    for i, j in enumerate(at):
        gk, bk, gv, bv = grads(p[:, i], G @ V[i], np.abs(G) @ np.abs(V[i]))
        assert (np.abs(A.f64(dk[j, 0]) - gk) <= bk).all() and (np.abs(A.f64(dv[j, 0]) - gv) <= bv).all(), j
    rest = torch.ones(lk, dtype=torch.bool, device="cuda")
    rest[at] = False
    gk, bk, gv, bv = grads(p0, 0.0, 0.0)
    for got, want, bound in ((dk, gk, bk), (dv, gv, bv)):
        # all zero keys have the same gradients: every one lies between the extremes of its column
        lo = torch.where(rest[:, None], got[:, 0], float("inf")).amin(0)
        hi = torch.where(rest[:, None], got[:, 0], float("-inf")).amax(0)
        assert (np.abs(A.f64(lo) - want) <= bound).all() and (np.abs(A.f64(hi) - want) <= bound).all()
        assert np.abs(want).min() > 0
    mag = np.abs(p * (G @ V.T - delta[:, None])) @ np.abs(K)
    want = scale * (p * (G @ V.T - delta[:, None])) @ K
    bound = u * np.abs(want) + scale * (mag * (u + 2 * ds) + (p * (err[:, None] + 2.0 ** -15 * (np.abs(G) @ np.abs(V).T)))
                                        @ np.abs(K)) + 2.0 ** -15 * scale * mag
    assert (np.abs(A.f64(dq[0]) - want) <= bound).all()


@pytest.mark.parametrize("hidden", [128, 300])
@pytest.mark.parametrize("lq,lk,Hq,Hk,D,dt", [(5, 700, 8, 1, 128, BF), (200, 900, 6, 2, 64, FP16), (40, 500, 2, 2, 128, FP16),
                                              (1, 9000, 8, 1, 128, BF), (150, 640, 32, 1, 64, BF)])
def test_first_keys_of_no_weight(lq, lk, Hq, Hk, D, dt, hidden):
    """The first keys a row sees score -inf (a key holds -inf) and weigh nothing: the result is that
    of the other keys alone, whatever their scores' size.

    Tolerances of out and lse as for any row: p's rounding and the output's (u), the score's error (2 ds),
    exponentials and sums (2^-18); fp16 loses p below 2^-25.
    """
    gen = torch.Generator().manual_seed(hidden + lq)
    r = lambda *s: torch.randn(*s, generator=gen).to(dt)  # noqa: E731
    q, k, v = r(lq, Hq, D), r(lk, Hk, D), r(lk, Hk, D)
    q[..., 0] = 1.0
    k[:hidden, :, 0] = float("-inf")
    scale, u, tiny = D ** -0.5, torch.finfo(dt).eps / 2, 2.0 ** -25 if dt == FP16 else 0.0
    for shift in (0.0, -400.0, 300.0):  # of all the other scores
        k[hidden:, :, 0] = shift / scale
        out, lse = csa.attn_forward(q.cuda(), k.cuda(), v.cuda(), _cu(lq), _cu(lk), scale)
        _ok()
        ref = A.attention(A.f64(q), A.f64(k[hidden:]), A.f64(v[hidden:]), [0, lq], [0, lk - hidden], scale)
        ds = 2.0 ** -16 * ref["smax"]
        err = np.abs(A.f64(out) - ref["out"])
        bound = u * np.abs(ref["out"]) + (u + 2 * ds[..., None] + 2.0 ** -18) * ref["mag_out"] + tiny * ref["vsum"]
        assert (err <= bound).all(), (shift, float((err / bound).max()))
        assert (np.abs(A.f64(lse) - ref["lse"]) <= ds + 2.0 ** -19 + 2.0 ** -22 * np.abs(ref["lse"])).all(), shift


@pytest.mark.parametrize("top", [17.3, 19.0])
@pytest.mark.parametrize("lq,lk,Hq,Hk,D", [(1, 131072, 8, 1, 128), (3, 60000, 2, 2, 64), (200, 20000, 4, 1, 64)])
def test_many_small_weights_in_fp16(lq, lk, Hq, Hk, D, top):
    """A dominant first key whose value is zero, and many keys whose weights are near or below 2^-25 of its own:
    the output is the sum of what those bring.

    u for p's rounding and for the output's, 2 ds for the score's error, 2^-18 for exponentials; the sum of
    weights adds up to a thousand tiles in fp32 (2^-24 each: 2^-14).  A weight below 2^-33 of the first tile's largest
    is lost.
    """
    gen = torch.Generator().manual_seed(lk)
    r = lambda *s: torch.randn(*s, generator=gen).to(FP16)  # noqa: E731
    q, k, v = r(lq, Hq, D), r(lk, Hk, D), 1 + 0.1 * r(lk, Hk, D)
    scale = D ** -0.5
    q[..., 0] = 1.0
    k[..., 0], k[0] = 0.0, 0.0
    k[0, :, 0], v[0] = top / scale, 0.0
    out, lse = csa.attn_forward(q.cuda(), k.cuda(), v.cuda(), _cu(lq), _cu(lk), scale)
    _ok()
    ref = A.attention(A.f64(q), A.f64(k), A.f64(v), [0, lq], [0, lk], scale)
    u, ds = 2.0 ** -11, 2.0 ** -16 * ref["smax"]
    err = np.abs(A.f64(out) - ref["out"])
    bound = (u * np.abs(ref["out"]) + (u + 2 * ds[..., None] + 2.0 ** -18 + 2.0 ** -14) * ref["mag_out"]
             + 2.0 ** -33 * ref["vsum"])
    assert (err <= bound).all(), float((err / bound).max())
    assert (np.abs(A.f64(lse) - ref["lse"]) <= ds + 2.0 ** -14 + 2.0 ** -22 * np.abs(ref["lse"])).all()


def _gradients(lq, lk, Hq, Hk, D, size, seed, vsize=1.0, qk=1.0):
    """(got, ref) of the fp16 gradients for cotangents of the given size; qk: size of q and k, at scores of unit size."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v = ((r(*s) * m).to(FP16) for s, m in (((sum(lq), Hq, D), qk), ((sum(lk), Hk, D), qk), ((sum(lk), Hk, D), vsize)))
    do = (r(sum(lq), Hq, D) * size).to(FP16)
    cu_q, cu_k, scale = _cu(*lq), _cu(*lk), D ** -0.5 / qk ** 2
    args = [t.cuda() for t in (q, k, v)]
    out, lse = csa.attn_forward(*args, cu_q, cu_k, scale)
    got = csa.attn_backward(do.cuda(), *args, out, lse, cu_q, cu_k, scale)
    _ok()
    ref = A.attention(A.f64(q), A.f64(k), A.f64(v), cu_q.cpu().numpy(), cu_k.cpu().numpy(), scale, dout=A.f64(do))
    return dict(zip(("dq", "dk", "dv"), got)), ref


@pytest.mark.parametrize("lq,lk,Hq,Hk,D", [([2, 1, 3], [2, 1, 3], 4, 4, 128), ([64, 40], [64, 90], 2, 2, 128),
                                           ([150], [400], 6, 2, 64), ([20], [9000], 4, 2, 64)])
def test_fp16_gradients_of_large_cotangents(lq, lk, Hq, Hk, D):
    """Cotangents of a scaled loss: p (dP - delta) passes fp16's range in places, the gradients do not.

    u for the rounding of p or ds and one of delta's, 2 ds, 2^-15 for the sums, u for the output's.
    """
    got, ref = _gradients(lq, lk, Hq, Hk, D, 2.0 ** 13, 7 * D + lk[0], vsize=3.0)
    u, top = 2.0 ** -11, 2.0 ** -15 * ref["smax"].max()
    for n in ("dq", "dk", "dv"):
        want = ref[n]
        assert np.abs(want).max() < 65000, n  # the inputs are chosen so
        bound = u * np.abs(want) + ((u if n == "dv" else 2 * u) + top + 2.0 ** -15) * ref["mag_" + n]
        err = np.abs(A.f64(got[n]) - want)
        assert (err <= bound + 2.0 ** -25).all(), (n, float((err / (bound + 2.0 ** -25)).max()))


@pytest.mark.parametrize("lq,lk,Hq,Hk,D,size", [([40], [6000], 4, 2, 64, 2.0 ** -10), ([30, 9], [4000, 2500], 2, 2, 128, 2.0 ** -12),
                                                ([300], [3000], 4, 1, 64, 2.0 ** -9)])
def test_fp16_gradients_of_small_cotangents(lq, lk, Hq, Hk, D, size):
    """Weights of 1/6000 times a small cotangent lie among fp16's last bits, if not below.

    Rounding errors are independent: in the root mean square each rounding (of ds, of delta's out, of the
    gradient) brings at most u, the scores 2 ds.  Small q and k at a large scale bring the gradients themselves
    among fp16's normal numbers.
    """
    got, ref = _gradients(lq, lk, Hq, Hk, D, size, lk[0], qk=2.0 ** -7)
    u, top = 2.0 ** -11, 2.0 ** -15 * ref["smax"].max()
    rms = lambda x: float(np.sqrt(np.mean(np.square(x))))  # noqa: E731
    for n in ("dq", "dk"):
        # the output's own last bit: 2^-25 where the gradient is below 2^-14
        assert rms(A.f64(got[n]) - ref[n]) <= (3 * u + top) * rms(ref[n]) + 2.0 ** -25, n


def test_fp16_gradients_of_many_small_weights():
    """dv of keys whose weight lies near 2^-20: p's rounding and the output's (u each), the score's error, and what
    a weight loses below 2^-40."""
    got, ref = _gradients([24], [200_000], 2, 1, 64, 2.0 ** 10, 5)
    u, top = 2.0 ** -11, 2.0 ** -15 * ref["smax"].max()
    err = np.abs(A.f64(got["dv"]) - ref["dv"])
    bound = u * np.abs(ref["dv"]) + (u + top + 2.0 ** -18) * ref["mag_dv"] + 2.0 ** -40 * ref["sum_dv"] + 2.0 ** -25
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("which", [0, 1, 2], ids=["dq", "dk", "dv"])
def test_each_gradient_by_differences(which):
    """sum(out * g) along the signs of the gradient's definition, so that all terms add up and the difference is
    far above its error: steps of 2^-5 and 2^-4 from a grid that fp16 holds.

    Values of out (below 4) and the weights in them are rounded to fp16 at independent points: 2^-10 / sqrt 3 each
    in the root mean square, six sigma over the step.  The curvature's error at the smaller step is a third of
    what the two steps differ by.  The gradient itself: four roundings of 2^-11 at most.
    """
    lq = [30, 21]
    gen = torch.Generator().manual_seed(29)
    x = [((torch.randn(51, h, 64, generator=gen)).clamp(-7, 7) * 128).round() / 128 for h in (4, 2, 2)]
    g = torch.randn(51, 4, 64, generator=gen).to(FP16)
    cu = _cu(*lq)
    ref = A.attention(*(A.f64(t) for t in x), cu.cpu().numpy(), cu.cpu().numpy(), 0.125, dout=A.f64(g))
    d = torch.from_numpy(np.sign(ref[("dq", "dk", "dv")[which]]))

    def value(s):
        y = [t.double() for t in x]
        y[which] = y[which] + s * d
        y16 = [t.to(FP16) for t in y]
        assert all(torch.equal(a.double(), b) for a, b in zip(y16, y))
        out, _ = csa.attn_forward(*(t.cuda() for t in y16), cu, cu, 0.125)
        return float((out.double().cpu() * g.double()).sum())

    base = [t.to(FP16).cuda() for t in x]
    out, lse = csa.attn_forward(*base, cu, cu, 0.125)
    got = csa.attn_backward(g.cuda(), *base, out, lse, cu, cu, 0.125)[which]
    _ok()
    along = float((got.double().cpu() * d).sum())
    h = 2.0 ** -5
    near, far = ((value(s) - value(-s)) / (2 * s) for s in (h, 2 * h))
    noise = 6 * 2 * float(g.double().norm()) * 2.0 ** -10 / 3 ** 0.5 / (2 * h)
    tol = noise + (abs(far - near) + noise) / 3 + 4 * 2.0 ** -11 * abs(near)
    assert tol < 0.02 * abs(near)  # zero, half or turned gradients would show
    assert abs(near - along) <= tol


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 60000.0])
def test_fp16_gradients_do_not_depend_on_other_sequences(bad):
    """dS's power of two comes from a sequence's own rows and keys: neighbours, and cache entries past the lengths,
    may hold anything; and the same call gives the same bits."""
    lq, W = [100, 37, 130, 60], 160
    gen = torch.Generator().manual_seed(51)
    r = lambda *s: torch.randn(*s, generator=gen).to(FP16)  # noqa: E731
    q, do, k, v = r(sum(lq), 8, 64), r(sum(lq), 8, 64), r(4 * W, 2, 64), r(4 * W, 2, 64)
    cu_q, cu_k, lens = _cu(*lq), _cu(*[W] * 4), torch.tensor([110, 37, 130, 90], dtype=torch.int32, device="cuda")

    def run():
        a = [t.cuda() for t in (q, k, v)]
        o = csa.attn_forward(*a, cu_q, cu_k, 0.125, k_len=lens)
        return (*o, *csa.attn_backward(do.cuda(), *a, *o, cu_q, cu_k, 0.125, k_len=lens))

    good, again = run(), run()
    assert all(torch.equal(a, b) for a, b in zip(good, again))
    rows, keys = torch.zeros(sum(lq), dtype=torch.bool), torch.arange(4 * W) // W == 1  # sequence 1
    rows[100:137] = True
    keys |= torch.arange(4 * W) % W >= lens.cpu().repeat_interleave(W)
    q[rows], do[rows], k[keys], v[keys] = bad, bad, bad, bad
    for i, (a, b) in enumerate(zip(good, run())):
        keep = ~(rows if i < 3 else keys).cuda()
        assert torch.equal(a[keep], b[keep])
    _ok()


def test_fp16_gradients_without_keys_or_sequences_and_in_a_graph():
    r = lambda *s: torch.randn(*s, generator=torch.Generator().manual_seed(s[0])).to(FP16).cuda()  # noqa: E731
    q, do, k, v = r(70, 6, 64), r(70, 6, 64), r(90, 2, 64), r(90, 2, 64)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kk, vv, cu_q, cu_k in ((k, v, none, none), (k[:0], v[:0], _cu(70), _cu(0)), (k, v, _cu(70, 0), _cu(0, 90))):
        out, lse = csa.attn_forward(q, kk, vv, cu_q, cu_k, 0.125)
        grads = csa.attn_backward(do, q, kk, vv, out, lse, cu_q, cu_k, 0.125)
        assert not out.any() and torch.isneginf(lse).all() and not any(g.any() for g in grads)
    cu_q, cu_k = _cu(30, 40), _cu(50, 40)
    step = lambda: csa.attn_backward(do, q, k, v, *csa.attn_forward(q, k, v, cu_q, cu_k, 0.125), cu_q, cu_k, 0.125)  # noqa: E731
    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):  # what a call leaves in its workspace does not reach the next
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    _ok()
