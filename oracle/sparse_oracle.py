"""Plain fp64 NumPy definition of attention over listed blocks of keys (test
infrastructure; imports nothing from the package).

Beside each result stands the sum of magnitudes its rounding errors scale with.
"""
import numpy as np


def counts(idx_rows, pos, lk, block, window, causal):
    """[rows, lk]: how often each row counts each key of its sequence."""
    n = np.zeros((len(pos), lk))
    for r, (row, at) in enumerate(zip(idx_rows, pos)):
        for b in row:
            if b < 0:
                continue
            for j in range(int(b) * block, min(lk, (int(b) + 1) * block)):
                if not causal or j <= at - window:
                    n[r, j] += 1
        if causal:
            n[r, max(0, at - window + 1):max(0, at + 1)] = 1 if window else n[r, max(0, at - window + 1):max(0, at + 1)]
    return n


def attention(q, k, v, idx, cu_q, cu_k, scale, block=1, window=0, causal=True, k_len=None, dout=None):
    """Forward, and with dout the gradients, of q [Tq,Hq,D], k, v [Tk,Hk,D], idx [Tq,top_k].

    Returns results and magnitudes under the names of attn_oracle.attention; "bound" [Tq,Hq] is
    2 scale max|dout| max|v| (2-norms, dout over the heads of a key head, v over the sequence), which
    |dout.v - dout.out| scale does not exceed; "norm_dk" and "norm_dv" [Tk,Hk] are sums over rows of
    scale m |q| and p |dout| with 2-norms (m: see there), what a row's share of a key is at most.
    """
    Tq, Hq, D = q.shape
    Hk = k.shape[1]
    g = Hq // Hk
    z = np.zeros
    res = dict(out=z(q.shape), lse=np.full((Tq, Hq), -np.inf), mag_out=z(q.shape), vsum=z(q.shape), smax=z((Tq, Hq)),
               bound=z((Tq, Hq)))
    if dout is not None:
        for n, like in (("dq", q), ("dk", k), ("dv", v)):
            res[n], res["mag_" + n], res["sum_" + n] = z(like.shape), z(like.shape), z(like.shape)
        res["norm_dk"], res["norm_dv"] = z(k.shape[:2]), z(k.shape[:2])
    for i in range(len(cu_q) - 1):
        a, b, c = int(cu_q[i]), int(cu_q[i + 1]), int(cu_k[i])
        lk = int(cu_k[i + 1]) - c if k_len is None else int(k_len[i])
        lq = b - a
        if lq == 0 or lk == 0:
            continue
        n = counts(idx[a:b], np.arange(lq) + lk - lq, lk, block, window, causal)
        see = n > 0
        any_ = see.any(1)
        for h in range(Hq):
            j = h // g
            Q, K, V = q[a:b, h], k[c:c + lk, j], v[c:c + lk, j]
            s = np.where(see, scale * (Q @ K.T), -np.inf)
            m = np.where(any_, np.max(s, axis=1, initial=-np.inf), 0.0)
            e = np.where(see, n * np.exp(s - m[:, None]), 0.0)
            l = e.sum(1)
            p = e / np.where(any_, l, 1.0)[:, None]
            o = p @ V
            res["out"][a:b, h] = o
            res["lse"][a:b, h] = np.where(any_, m + np.log(np.where(any_, l, 1.0)), -np.inf)
            res["mag_out"][a:b, h] = p @ np.abs(V)
            res["vsum"][a:b, h] = n @ np.abs(V)
            res["smax"][a:b, h] = np.where(see, scale * (np.abs(Q) @ np.abs(K).T), 0.0).max(1)
            if dout is None:
                continue
            G = dout[a:b, h]
            most = np.linalg.norm(dout[a:b, j * g:(j + 1) * g], axis=2).max(1)
            res["bound"][a:b, h] = 2 * scale * most * np.linalg.norm(V, axis=1).max()
            dp = G @ V.T
            ds = p * (dp - (G * o).sum(1, keepdims=True))
            dmag = np.abs(ds) + p * ((np.abs(G) * np.abs(o)).sum(1, keepdims=True) + np.abs(G) @ np.abs(V).T)
            top = n * res["bound"][a:b, h][:, None]
            res["dq"][a:b, h] = scale * (ds @ K)
            res["mag_dq"][a:b, h] = scale * (dmag @ np.abs(K))
            res["sum_dq"][a:b, h] = top @ np.abs(K)
            res["dk"][c:c + lk, j] += scale * (ds.T @ Q)
            res["mag_dk"][c:c + lk, j] += scale * (dmag.T @ np.abs(Q))
            res["sum_dk"][c:c + lk, j] += top.T @ np.abs(Q)
            res["dv"][c:c + lk, j] += p.T @ G
            res["mag_dv"][c:c + lk, j] += p.T @ np.abs(G)
            res["sum_dv"][c:c + lk, j] += n.T @ np.abs(G)
            res["norm_dk"][c:c + lk, j] += scale * (dmag.T @ np.linalg.norm(Q, axis=1))
            res["norm_dv"][c:c + lk, j] += p.T @ np.linalg.norm(G, axis=1)
    return res
