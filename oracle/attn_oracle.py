"""Plain fp64 NumPy definitions of the norm + rotation and of packed attention
(test infrastructure; imports nothing from the package).

Beside each result stands the sum of magnitudes its rounding errors scale
with, so that tests can state their tolerances before they run.
"""
import numpy as np


def f64(t):
    """Exact float64 copy of a tensor of any storage type."""
    import torch

    return t.detach().to(torch.float64).cpu().numpy()


# ----------------------------------------------------------------------------- norm + rotation
def _pairs(D, rot, off, interleaved):
    """Indices (u, v) of the turned pairs."""
    i = np.arange(rot // 2)
    return (off + 2 * i, off + 2 * i + 1) if interleaved else (off + i, off + rot // 2 + i)


def _turn(x, ang, rot, off, interleaved, back=False):
    """x [T,H,D] with its pairs turned by ang [T,rot/2]; and the magnitudes |u cos| + |v sin| of each value."""
    u, v = _pairs(x.shape[-1], rot, off, interleaved)
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :] * (-1.0 if back else 1.0)
    y, mag = x.copy(), np.abs(x)
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., u] * s + x[..., v] * c
    mag[..., u] = mag[..., v] = np.abs(x[..., u]) + np.abs(x[..., v])
    return y, mag


def norm_rope(x, w, ang, eps, off, interleaved):
    """(y, magnitudes) of x [T,H,D]; ang [T,rot/2] in radians."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _turn(x * r * w, ang, 2 * ang.shape[1], off, interleaved)


def norm_rope_vjp(dy, x, w, ang, eps, off, interleaved):
    """(dx, magnitudes of dx, dw, magnitudes of dw)."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    z, zmag = _turn(dy, ang, 2 * ang.shape[1], off, interleaved, back=True)
    dn = z * w
    dx = r * (dn - xh * (dn * xh).mean(-1, keepdims=True))
    mag = r * (zmag * np.abs(w) + np.abs(xh) * (zmag * np.abs(w * xh)).mean(-1, keepdims=True))
    return dx, mag, (z * xh).sum((0, 1)), (zmag * np.abs(xh)).sum((0, 1))


# ----------------------------------------------------------------------------- attention
def visible(lq, lk, causal=True):
    """[lq,lk]: which keys each row sees (the last query stands at the last key)."""
    if not causal:
        return np.ones((lq, lk), dtype=bool)
    return np.arange(lk)[None, :] <= np.arange(lq)[:, None] + lk - lq


def attention(q, k, v, cu_q, cu_k, scale, causal=True, k_len=None, dout=None):
    """Forward, and with dout the gradients, of q [Tq,Hq,D], k, v [Tk,Hk,D].

    Returns a dict of results and, under "mag_*", the sums of magnitudes:
      mag_out = sum p |v|,  smax = largest scale*|q|.|k| of the row (scores' error scales with it),
      mag_dv = sum p |dout|,  mag_dq / mag_dk = scale * sum over terms of m |k| (|q|) with
      m = |ds| + p (sum |dout||out| + |dout|.|v|): ds's own rounding and the errors of delta and dout.v.
    """
    Tq, Hq, D = q.shape
    Tk, Hk, _ = k.shape
    g = Hq // Hk
    z = np.zeros
    res = dict(out=z(q.shape), lse=np.full((Tq, Hq), -np.inf), mag_out=z(q.shape), vsum=z(q.shape), smax=z((Tq, Hq)))
    if dout is not None:
        for n, like in (("dq", q), ("dk", k), ("dv", v)):
            res[n], res["mag_" + n], res["sum_" + n] = z(like.shape), z(like.shape), z(like.shape)
    for i in range(len(cu_q) - 1):
        a, b, c = int(cu_q[i]), int(cu_q[i + 1]), int(cu_k[i])
        lk = int(cu_k[i + 1]) - c if k_len is None else int(k_len[i])
        lq = b - a
        if lq == 0 or lk == 0:
            continue
        see = visible(lq, lk, causal)
        any_ = see.any(1)
        for h in range(Hq):
            j = h // g
            Q, K, V = q[a:b, h], k[c:c + lk, j], v[c:c + lk, j]
            s = np.where(see, scale * (Q @ K.T), -np.inf)
            m = np.where(any_, np.max(s, axis=1, initial=-np.inf), 0.0)
            e = np.where(see, np.exp(s - m[:, None]), 0.0)
            l = e.sum(1)
            p = e / np.where(any_, l, 1.0)[:, None]
            o = p @ V
            res["out"][a:b, h] = o
            res["lse"][a:b, h] = np.where(any_, m + np.log(np.where(any_, l, 1.0)), -np.inf)
            res["mag_out"][a:b, h] = p @ np.abs(V)
            res["vsum"][a:b, h] = see.astype(float) @ np.abs(V)
            smag = np.where(see, scale * (np.abs(Q) @ np.abs(K).T), 0.0)
            res["smax"][a:b, h] = smag.max(1)
            if dout is None:
                continue
            G = dout[a:b, h]
            dp = G @ V.T
            ds = p * (dp - (G * o).sum(1, keepdims=True))
            dmag = np.abs(ds) + p * ((np.abs(G) * np.abs(o)).sum(1, keepdims=True) + np.abs(G) @ np.abs(V).T)
            sf = see.astype(float)
            res["dq"][a:b, h] = scale * (ds @ K)
            res["mag_dq"][a:b, h] = scale * (dmag @ np.abs(K))
            res["sum_dq"][a:b, h] = scale * (sf @ np.abs(K))
            res["dk"][c:c + lk, j] += scale * (ds.T @ Q)
            res["mag_dk"][c:c + lk, j] += scale * (dmag.T @ np.abs(Q))
            res["sum_dk"][c:c + lk, j] += scale * (sf.T @ np.abs(Q))
            res["dv"][c:c + lk, j] += p.T @ G
            res["mag_dv"][c:c + lk, j] += p.T @ np.abs(G)
            res["sum_dv"][c:c + lk, j] += sf.T @ np.abs(G)
    return res
