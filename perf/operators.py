"""Cases of the operators around the indexer: the norm and rotation of queries and
keys, and causal attention over packed sequences, each in its plain form (elementary
torch operations in 32 bits) and as calls of the library.

Every case is one pass of one operator.  `own` chooses which form `run` takes.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
THETA = 10000.0


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 sequences at the end of a 131072-token context: the smallest call, all latency
        dict(name="norm_rope_token", op="norm_rope", T=64, Hq=64, Hk=8, D=128, rot=128, off=0, inter=False,
             dtype="bf16", wtype="bf16", pos=131071, doc=0, train=False),
        # a prompt of 16384 tokens, 64 query and 8 key heads of 128
        dict(name="norm_rope_prompt", op="norm_rope", T=16384, Hq=64, Hk=8, D=128, rot=128, off=0, inter=False,
             dtype="bf16", wtype="bf16", pos=0, doc=0, train=False),
        # odd token count, 32-bit data, the small heads of 32, neighbouring pairs, half of each head turned, far positions
        dict(name="norm_rope_odd", op="norm_rope", T=4099, Hq=12, Hk=3, D=32, rot=16, off=16, inter=True,
             dtype="fp32", wtype="fp32", pos=900001, doc=0, train=False),
        # a training step on 4 x 8192 packed tokens (positions restart with each document)
        dict(name="norm_rope_train", op="norm_rope", T=32768, Hq=64, Hk=8, D=128, rot=64, off=64, inter=True,
             dtype="bf16", wtype="bf16", pos=0, doc=1500, train=True),
        # a small training step with odd sizes, fp16, weights kept in 32 bits
        dict(name="norm_rope_train_odd", op="norm_rope", T=1537, Hq=15, Hk=5, D=64, rot=64, off=0, inter=False,
             dtype="fp16", wtype="fp32", pos=0, doc=257, train=True),
        # one whole prompt of 16384 tokens: the largest case
        dict(name="attn_prompt", op="attn", T=16384, docs=1, Hq=64, Hk=8, D=128, dtype="bf16", prefix=0, ragged=False,
             train=False),
        # 4 x 8192 tokens of packed documents, three to eight in each row of 8192
        dict(name="attn_packed", op="attn", T=32768, docs=22, Hq=64, Hk=8, D=128, dtype="bf16", prefix=0, ragged=False,
             train=False),
        # many short pieces of odd lengths, empty ones and single tokens among them, some behind a cached prefix and
        # some with fewer keys than queries (rows that see nothing)
        dict(name="attn_short", op="attn", T=2011, docs=41, Hq=12, Hk=4, D=64, dtype="fp16", prefix=333, ragged=True,
             train=False),
        # forward and backward of a training step on 8192 packed tokens
        dict(name="attn_train", op="attn", T=8192, docs=5, Hq=64, Hk=8, D=128, dtype="bf16", prefix=0, ragged=False,
             train=True),
        # a small training step: odd lengths, three query heads to a key head, fp16, heads of 64
        dict(name="attn_train_odd", op="attn", T=1021, docs=6, Hq=9, Hk=3, D=64, dtype="fp16", prefix=0, ragged=True,
             train=True),
        # one token of each of 64 sequences over a cache of up to 8192 entries, lengths from a quarter to full
        dict(name="attn_decode", op="decode", N=64, W=8192, Hq=64, Hk=8, D=128, dtype="bf16"),
        # one token of a single sequence over 131072 cached entries: the long axis has to be split
        dict(name="attn_decode_long", op="decode", N=1, W=131072, Hq=64, Hk=8, D=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm_rope", "norm_rope_train", "attn", "attn_train", "decode"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind.startswith("norm_rope"):
        D = rng.choice([32, 64, 128])
        rot = rng.choice([r for r in (16, 32, 64, 128) if r <= D])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        g = rng.choice([1, 3, 4, 8])
        Hk = rng.choice([1, 2, 5, 8])
        T = min(_log(rng, 1, 32768), 32768 * 64 * 128 // (g * Hk * D) // 4)
        return dict(op="norm_rope", T=max(1, T), Hq=g * Hk, Hk=Hk, D=D, rot=rot, off=rng.choice([0, D - rot]),
                    inter=rng.random() < 0.5, dtype=dtype, wtype=rng.choice([dtype, "fp32"]),
                    pos=_log(rng, 1, 1000000), doc=rng.choice([0, _log(rng, 7, 5000)]),
                    train=kind.endswith("train"))
    D = rng.choice([64, 128])
    g = rng.choice([1, 3, 4, 8, 16])
    Hk = rng.choice([1, 2, 4, 8]) if g < 16 else rng.choice([1, 2, 4])
    if kind == "decode":
        N = _log(rng, 1, 128)
        W = min(_log(rng, 17, 131072), 131072 * 8 // (N * Hk))
        return dict(op="decode", N=N, W=max(17, W), Hq=g * Hk, Hk=Hk, D=D, dtype=dtype)
    T = _log(rng, 60, 8192 if kind == "attn_train" else 16384)
    return dict(op="attn", T=T, docs=_log(rng, 1, max(1, T // 20)) if T > 40 else 1, Hq=g * Hk, Hk=Hk, D=D, dtype=dtype,
                prefix=rng.choice([0, _log(rng, 1, 2000)]), ragged=rng.random() < 0.5, train=kind == "attn_train")


# ----------------------------------------------------------------------------- inputs
def _lengths(case):
    """Query and key lengths of the packed sequences of an attention case (host lists): the case's own, so that
    every seed's tensors have the same shapes."""
    T, n = case["T"], case["docs"]
    rng = np.random.default_rng(T * 7919 + n)
    cuts = np.sort(rng.integers(1, T, n - 1)) if n > 1 else np.array([], dtype=np.int64)
    if case["ragged"] and n > 4:
        cuts[1] = cuts[0]          # an empty sequence
        cuts[3] = cuts[2] + 1      # a single token
        cuts = np.sort(np.minimum(cuts, T))
    lq = np.diff(np.concatenate([[0], cuts, [T]])).astype(np.int64)
    lk = lq.copy()
    if case["prefix"]:             # keys of earlier tokens in front of some sequences
        lk = lk + rng.integers(0, case["prefix"] + 1, n) * rng.integers(0, 2, n)
    if case["ragged"] and not case["train"]:
        short = rng.integers(0, 6, n) == 0   # fewer keys than queries: the first rows see nothing
        lk = np.where(short, lk // 2, lk)
    if lk.sum() == 0:
        lk[0] = 1
    return [int(x) for x in lq], [int(x) for x in lk]


def _decode_lengths(case, seed):
    rng = np.random.default_rng(seed * 104729 + 5)
    W = case["W"]
    length = rng.integers(max(1, W // 4), W + 1, case["N"])
    length[0] = W
    return [int(x) for x in length]


def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    if case["op"] == "norm_rope":
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        st = dict(case)
        # q and k as they leave the projection: views of one wider row, of uneven size per head
        qkv = randn(T, Hq + 2 * Hk, D) * torch.exp(0.5 * randn(1, Hq + 2 * Hk, 1, dtype=torch.float32)).to(dt)
        st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        wt = DTYPES[case["wtype"]]
        st["qw"] = (1 + 0.2 * randn(D, dtype=torch.float32)).to(wt)
        st["kw"] = (1 + 0.2 * randn(D, dtype=torch.float32)).to(wt)
        if T <= 64 and case["pos"]:
            st["pos"] = torch.full((T,), case["pos"], dtype=torch.int64, device="cuda") - torch.randint(
                0, case["pos"], (T,), generator=gen, device="cuda") // 2
        else:
            p = torch.arange(T, device="cuda")
            st["pos"] = case["pos"] + (p % case["doc"] if case["doc"] else p)
        if case["train"]:
            st["dqo"], st["dko"] = randn(T, Hq, D), randn(T, Hk, D)
        st["inv"] = THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        st["freqs"] = _freqs(case["rot"])
        return st
    st = dict(case)
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    st["scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "decode":
        N, W = case["N"], case["W"]
        st["q"] = randn(N, Hq, D)
        st["k"], st["v"] = randn(N * W, Hk, D), randn(N * W, Hk, D)
        st["cu_q"] = torch.arange(N + 1, dtype=torch.int32, device="cuda")
        st["cu_k"] = st["cu_q"] * W
        st["k_len"] = torch.tensor(_decode_lengths(case, seed), dtype=torch.int32, device="cuda")
        return st
    lq, lk = _lengths(case)
    st["lq"], st["lk"] = lq, lk
    st["q"] = randn(sum(lq), Hq, D)
    kv = randn(sum(lk), 2 * Hk, D)
    st["k"], st["v"] = kv[:, :Hk], kv[:, Hk:]
    st["cu_q"], st["cu_k"] = _cu(lq), _cu(lk)
    if case["train"]:
        st["dout"] = randn(sum(lq), Hq, D)
    return st


def _freqs(rot):
    """Turns per position of each pair as 64-bit fixed-point fractions: the table that the library's calls take."""
    turns = [int(round(THETA ** (-i / rot) / (2 * math.pi) * 2.0 ** 64)) for i in range(0, rot, 2)]
    return torch.tensor(np.array(turns, dtype=np.uint64).view(np.int64), device="cuda")


# ----------------------------------------------------------------------------- plain forms
def _angles(st):
    """cos and sin [T, rot/2] of the pairs' angles, from 64-bit products (far positions)."""
    a = st["pos"].to(torch.float64)[:, None] * st["inv"][None, :]
    return torch.cos(a).float(), torch.sin(a).float()


def _halves(x, st):
    """The two members of each turned pair, as views [T, H, rot/2]."""
    z = x[..., st["off"]:st["off"] + st["rot"]]
    if st["inter"]:
        return z[..., 0::2], z[..., 1::2]
    return z[..., :st["rot"] // 2], z[..., st["rot"] // 2:]


def _turn(x, cos, sin, st):
    """x with its pairs turned by the angles (in place on a fresh 32-bit tensor)."""
    a, b = _halves(x, st)
    na, nb = a * cos[:, None] - b * sin[:, None], a * sin[:, None] + b * cos[:, None]
    a.copy_(na)
    b.copy_(nb)
    return x


def _norm_rope_plain(x, w, cos, sin, st):
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    return _turn(x32 * r * w.float(), cos, sin, st).to(x.dtype)


def _norm_rope_grad_plain(dy, x, w, cos, sin, st):
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    xh = x32 * r
    dz = _turn(dy.float().clone(), cos, -sin, st)
    dw = (dz * xh).sum((0, 1))
    dn = dz * w.float()
    return (r * (dn - xh * (dn * xh).mean(-1, keepdim=True))).to(x.dtype), dw


def _visible(st, q0, q1):
    """Key range [k0, k1) that the query rows [q0, q1) can see, and the mask [q1-q0, k1-k0] of what each sees."""
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    cq, ck = np.concatenate([[0], np.cumsum(st["lq"])]), np.concatenate([[0], np.cumsum(st["lk"])])
    a, b = np.searchsorted(cq, q0, "right") - 1, np.searchsorted(cq, q1 - 1, "right") - 1
    end = int(ck[b + 1] - max(0, cq[b + 1] - q1)) if a == b else int(ck[b + 1])
    k0 = min(int(ck[a]), int(ck[-1]) - 1)
    k1 = max(end, k0 + 1)   # one hidden key at least, so that no dimension is empty
    rows = torch.arange(q0, q1, device="cuda")
    keys = torch.arange(k0, k1, device="cuda")
    sq = torch.searchsorted(cu_q, rows, right=True) - 1
    last = cu_k[sq + 1] - (cu_q[sq + 1] - rows)
    return k0, k1, (keys[None] >= cu_k[sq][:, None]) & (keys[None] <= last[:, None])


def _scores(q, k, mask, scale):
    """Masked scores [Hk, g, rows, keys]."""
    R, Hq, D = q.shape
    Hk = k.shape[1]
    q32 = q.float().reshape(R, Hk, Hq // Hk, D).permute(1, 2, 0, 3).reshape(Hk, -1, D)
    s = (q32 @ k.float().permute(1, 2, 0)) * scale
    return s.reshape(Hk, Hq // Hk, R, -1).masked_fill_(~mask, -math.inf), q32


def _by_heads(x, Hk):
    """[rows, Hq, D] as [Hk, g * rows, D] in 32 bits."""
    R, Hq, D = x.shape
    return x.float().reshape(R, Hk, Hq // Hk, D).permute(1, 2, 0, 3).reshape(Hk, -1, D)


def _by_rows(x, R):
    """[Hk, g * rows, D] as [rows, Hq, D]."""
    Hk, _, D = x.shape
    return x.reshape(Hk, -1, R, D).permute(2, 0, 1, 3).reshape(R, -1, D)


def _attn_plain(st):
    """Forward (and gradients) in blocks of query rows: all scores of a long prompt would not fit the card."""
    q, k, v, scale = st["q"], st["k"], st["v"], st["scale"]
    T, Hq, D = q.shape
    Hk = k.shape[1]
    step = max(16, min(T, (1 << 28) // (Hq * max(1, k.shape[0]))))
    out = torch.zeros_like(q)
    lse = torch.full((T, Hq), -math.inf, device="cuda")
    if st["train"]:
        dq = torch.zeros_like(q)
        dk = torch.zeros(k.shape, device="cuda")
        dv = torch.zeros(v.shape, device="cuda")
    for q0 in range(0, T, step):
        q1 = min(T, q0 + step)
        R = q1 - q0
        k0, k1, mask = _visible(st, q0, q1)
        s, q32 = _scores(q[q0:q1], k[k0:k1], mask, scale)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
        l = p.sum(-1, keepdim=True)
        p = (p / torch.where(l == 0, 1.0, l)).reshape(Hk, -1, k1 - k0)
        o = p @ v[k0:k1].float().permute(1, 0, 2)
        out[q0:q1] = _by_rows(o, R).to(q.dtype)
        lse[q0:q1] = (m + torch.log(l))[..., 0].permute(2, 0, 1).reshape(R, Hq)
        if st["train"]:
            do = _by_heads(st["dout"][q0:q1], Hk)
            dv[k0:k1] += (p.transpose(1, 2) @ do).permute(1, 0, 2)
            dp = do @ v[k0:k1].float().permute(1, 2, 0)
            ds = p * (dp - (do * o).sum(-1, keepdim=True)) * scale
            dq[q0:q1] = _by_rows(ds @ k[k0:k1].float().permute(1, 0, 2), R).to(q.dtype)
            dk[k0:k1] += (ds.transpose(1, 2) @ q32).permute(1, 0, 2)
    if st["train"]:
        return dict(out=out, lse=lse, dq=dq, dk=dk.to(k.dtype), dv=dv.to(v.dtype))
    return dict(out=out, lse=lse)


def _decode_plain(st):
    q, scale = st["q"], st["scale"]
    N, Hq, D = q.shape
    W, Hk = st["W"], st["Hk"]
    k32 = st["k"].float().reshape(N, W, Hk, D).permute(0, 2, 3, 1)
    v32 = st["v"].float().reshape(N, W, Hk, D).permute(0, 2, 1, 3)
    s = (q.float().reshape(N, Hk, Hq // Hk, D) @ k32) * scale
    s = s.masked_fill_((torch.arange(W, device="cuda") >= st["k_len"][:, None])[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    out = ((p / l) @ v32).reshape(N, Hq, D).to(q.dtype)
    return dict(out=out, lse=(m + torch.log(l)).reshape(N, Hq))


# ----------------------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "norm_rope":
        cos, sin = _angles(st)
        res = dict(q_out=_norm_rope_plain(st["q"], st["qw"], cos, sin, st),
                   k_out=_norm_rope_plain(st["k"], st["kw"], cos, sin, st))
        if st["train"]:
            res["dq"], res["dqw"] = _norm_rope_grad_plain(st["dqo"], st["q"], st["qw"], cos, sin, st)
            res["dk"], res["dkw"] = _norm_rope_grad_plain(st["dko"], st["k"], st["kw"], cos, sin, st)
        return res
    return _decode_plain(st) if st["op"] == "decode" else _attn_plain(st)


def _run_own(st):
    import sparse_attention_indexer_csa_gb300 as csa

    if st["op"] == "norm_rope":
        kw = dict(eps=EPS, rot_offset=st["off"], interleaved=st["inter"])
        q_out, k_out = csa.norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["pos"], st["freqs"], **kw)
        if not st["train"]:
            return dict(q_out=q_out, k_out=k_out)
        dq, dk, dqw, dkw = csa.norm_rope_backward(st["dqo"], st["dko"], st["q"], st["k"], st["qw"], st["kw"],
                                                  st["pos"], st["freqs"], **kw)
        return dict(q_out=q_out, k_out=k_out, dq=dq, dqw=dqw, dk=dk, dkw=dkw)
    out, lse = csa.attn_forward(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], st["scale"],
                                k_len=st.get("k_len"))
    if not st.get("train"):
        return dict(out=out, lse=lse)
    dq, dk, dv = csa.attn_backward(st["dout"], st["q"], st["k"], st["v"], out, lse, st["cu_q"], st["cu_k"],
                                   st["scale"])
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


# ----------------------------------------------------------------------------- what a pass cannot do without
def _pairs(lq, lk):
    """Visible (query, key) pairs of one sequence, the last query aligned with the last key."""
    return lq * lk - lq * (lq - 1) // 2 if lq <= lk else lk * (lk + 1) // 2


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if case["op"] == "norm_rope":
        n = case["T"] * (Hq + Hk) * D
        we = 4 if case["wtype"] == "fp32" else 2
        small = case["T"] * 8 + 2 * D * we + case["rot"] * 4
        if case["train"]:   # x and dy in, y and dx out, two weight gradients
            return dict(bytes=4 * n * e + small + 8 * D, flops=20 * n)
        return dict(bytes=2 * n * e + small, flops=8 * n)
    if case["op"] == "decode":
        n = sum(_decode_lengths(case, 0))
        N = case["N"]
        return dict(bytes=2 * n * Hk * D * e + 2 * N * Hq * D * e + N * Hq * 4 + 12 * N, flops=4 * n * Hq * D)
    lq, lk = _lengths(case)
    pairs = sum(_pairs(a, b) for a, b in zip(lq, lk)) * Hq
    nq, nk = sum(lq) * Hq * D * e, sum(lk) * Hk * D * e
    small = sum(lq) * Hq * 4 + 8 * len(lq)
    if case["train"]:
        return dict(bytes=4 * nq + 4 * nk + small, flops=14 * D * pairs)
    return dict(bytes=2 * nq + 2 * nk + small, flops=4 * D * pairs)


# ----------------------------------------------------------------------------- the definition in 64 bits
def _exact_norm_rope(st):
    """Norm and rotation as products of complex numbers; gradients by differentiating the definition."""
    pos, rot, off = st["pos"].double(), st["rot"], st["off"]
    expo = torch.arange(rot // 2, dtype=torch.float64, device="cuda") * (-2.0 / rot)
    unit = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                       pos.unsqueeze(1) * torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"), expo))

    def turned(x, w):
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
        body = y[..., off:off + rot]
        pairs = body.unflatten(-1, (rot // 2, 2)) if st["inter"] else body.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_complex(pairs.contiguous()) * unit[:, None, :]
        flat = torch.view_as_real(z)
        flat = flat.flatten(-2) if st["inter"] else flat.transpose(-1, -2).flatten(-2)
        return torch.cat([y[..., :off], flat, y[..., off + rot:]], -1)

    res = {}
    parts = [("q_out", "dq", "dqw", st["q"], st["qw"], st.get("dqo")), ("k_out", "dk", "dkw", st["k"], st["kw"], st.get("dko"))]
    for y_name, dx_name, dw_name, x, w, dy in parts:
        T, H, D = x.shape
        w64 = w.double().requires_grad_(st["train"])
        y = torch.empty(T, H, D, dtype=torch.float64, device="cuda")
        dx = torch.empty_like(y) if st["train"] else None
        dw = torch.zeros(D, dtype=torch.float64, device="cuda")
        for h in range(H):   # a head at a time bounds the memory of the graph
            x64 = x[:, h:h + 1].double().requires_grad_(st["train"])
            yh = turned(x64, w64)
            y[:, h:h + 1] = yh.detach()
            if st["train"]:
                gx, gw = torch.autograd.grad(yh, (x64, w64), dy[:, h:h + 1].double())
                dx[:, h:h + 1] = gx
                dw += gw
        res[y_name] = y
        if st["train"]:
            res[dx_name], res[dw_name] = dx, dw
    names = ("q_out", "k_out", "dq", "dqw", "dk", "dkw") if st["train"] else ("q_out", "k_out")
    return {n: res[n] for n in names}


def _exact_one(q, k, v, scale, first, dout=None):
    """One head of one sequence: row i sees keys 0 .. first + i.  Gradients by differentiating the definition."""
    leaves = [t.double() for t in (q, k, v)]
    if dout is not None:
        leaves = [t.requires_grad_(True) for t in leaves]
    q64, k64, v64 = leaves
    s = torch.matmul(q64, k64.T) * scale
    hidden = torch.arange(k.shape[0], device="cuda")[None] > first + torch.arange(q.shape[0], device="cuda")[:, None]
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    o = torch.matmul(torch.exp(s - lse[:, None]), v64)
    if dout is None:
        return o, lse, ()
    return o.detach(), lse.detach(), torch.autograd.grad(o, leaves, dout.double())


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_norm_rope(st)
    Hq, Hk, D, scale = case["Hq"], case["Hk"], case["D"], st["scale"]
    g = Hq // Hk
    T = st["q"].shape[0]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    if case["op"] == "decode":
        W = case["W"]
        for n, length in enumerate(_decode_lengths(case, seed)):
            for j in range(Hk):
                rows = slice(n * W, n * W + length)
                h = slice(j * g, (j + 1) * g)
                s = st["k"][rows, j].double() @ st["q"][n, h].double().T * scale
                lse[n, h] = torch.logsumexp(s, 0)
                out[n, h] = torch.softmax(s, 0).T @ st["v"][rows, j].double()
        return dict(out=out, lse=lse)
    grads = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in (st["q"], st["k"], st["v"])]
    a = c = 0
    for lq, lk in zip(st["lq"], st["lk"]):
        n = min(lq, lk)          # the rows that see a key
        for h in range(Hq if n else 0):
            j = h // g
            for r0 in range(lq - n, lq, 4096):
                r1 = min(lq, r0 + 4096)
                seen = lk - lq + r1
                rows, keys = slice(a + r0, a + r1), slice(c, c + seen)
                o, l, gr = _exact_one(st["q"][rows, h], st["k"][keys, j], st["v"][keys, j], scale, lk - lq + r0,
                                      st["dout"][rows, h] if case["train"] else None)
                out[rows, h], lse[rows, h] = o, l
                if gr:
                    grads[0][rows, h] += gr[0]
                    grads[1][keys, j] += gr[1]
                    grads[2][keys, j] += gr[2]
        a, c = a + lq, c + lk
    if not case["train"]:
        return dict(out=out, lse=lse)
    return dict(out=out, lse=lse, dq=grads[0], dk=grads[1], dv=grads[2])
