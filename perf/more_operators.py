"""Cases of the operators that use the indexer's selection and the cache they read: norm and rotation with an
append to a paged cache, attention over listed blocks of keys with its gradients, and the same attention over the
paged cache for single tokens.  Each in its plain form (elementary torch operations in 32 bits) and as calls of the
library.

Every case is one pass of one operator (a training case: forward and gradients).  `own` chooses which form `run`
takes.
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
        # one token of each of 64 sequences, put behind 131 to 250 cached ones: the smallest call, all latency
        dict(name="append_token", op="append", N=64, T=64, past=250, page=64, Hq=64, Hk=8, D=128, rot=128, off=0,
             inter=False, dtype="bf16", wtype="bf16"),
        # a prompt of 16384 tokens in three sequences, the first pages of an empty cache
        dict(name="append_prompt", op="append", N=3, T=16384, past=0, page=64, Hq=64, Hk=8, D=128, rot=64, off=64,
             inter=True, dtype="bf16", wtype="bf16"),
        # odd counts, pages of 24, a chunk of each prompt behind what is cached, half of each head turned
        dict(name="append_odd", op="append", N=11, T=1537, past=301, page=24, Hq=15, Hk=5, D=64, rot=32, off=32,
             inter=False, dtype="fp16", wtype="fp32"),
        # a prompt of 16384 tokens over its 4096 compressed entries, 512 kept per row: the indexer's own shape
        dict(name="sparse_prompt", op="sparse", T=16384, docs=1, Hq=64, Hk=1, D=128, K=512, block=1, window=0, rate=4,
             prefix=0, ragged=False, dtype="bf16", train=False),
        # the tokens that the kept entries stand for, and the last 128: two prompts, 16 query heads to a key head
        dict(name="sparse_tokens", op="sparse", T=8192, docs=2, Hq=32, Hk=2, D=128, K=256, block=4, window=128, rate=0,
             prefix=0, ragged=False, dtype="bf16", train=False),
        # short pieces of odd lengths, empty ones and single tokens among them, some behind cached keys and some with
        # fewer keys than queries (rows that see nothing), odd lists and windows
        dict(name="sparse_odd", op="sparse", T=1021, docs=13, Hq=9, Hk=3, D=64, K=77, block=2, window=33, rate=0,
             prefix=200, ragged=True, dtype="fp16", train=False),
        # forward and gradients of 8192 tokens over their 2048 entries, 256 kept
        dict(name="sparse_train", op="sparse", T=8192, docs=1, Hq=64, Hk=1, D=128, K=256, block=1, window=0, rate=4,
             prefix=0, ragged=False, dtype="bf16", train=True),
        # the same with larger blocks of tokens and a window, packed documents, 16 query heads to a key head
        dict(name="sparse_train_blocks", op="sparse", T=4096, docs=3, Hq=32, Hk=2, D=128, K=16, block=16, window=64,
             rate=0, prefix=0, ragged=False, dtype="bf16", train=True),
        # a small training step with odd sizes, fp16, heads of 64
        dict(name="sparse_train_odd", op="sparse", T=517, docs=5, Hq=10, Hk=2, D=64, K=19, block=4, window=7, rate=0,
             prefix=0, ragged=True, dtype="fp16", train=True),
        # one token of each of 64 sequences over a paged cache of 8192 to 32768 tokens: 512 blocks of 4 and the last 128
        dict(name="paged_decode", op="paged", N=64, nq=1, W=32768, page=64, Hq=64, Hk=8, D=128, K=512, block=4,
             window=128, dtype="bf16"),
        # one token of a single sequence of 131072 tokens: few rows, the list has to be split
        dict(name="paged_decode_long", op="paged", N=1, nq=1, W=131072, page=64, Hq=64, Hk=8, D=128, K=512, block=4,
             window=128, dtype="bf16"),
        # three tokens of each of seven sequences (a draft that is checked), pages of 24, odd lists, heads of 64
        dict(name="paged_odd", op="paged", N=7, nq=3, W=2001, page=24, Hq=12, Hk=4, D=64, K=93, block=2, window=17,
             dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(["append", "sparse", "sparse_train", "paged"])
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([64, 128])
    g = rng.choice([1, 3, 4, 8, 16, 32, 64, 128])
    Hk = rng.choice([1, 2, 4, 8]) if g <= 16 else rng.choice([1, 2]) if g <= 64 else 1
    if kind == "append":
        Hk, g = rng.choice([1, 2, 5, 8]), rng.choice([1, 3, 4, 8])
        D = rng.choice([32, 64, 128])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        rot = rng.choice([r for r in (16, 32, 64, 128) if r <= D])
        T = max(1, min(_log(rng, 1, 16384), 16384 * 72 * 128 // ((g + 2) * Hk * D)))
        return dict(op="append", N=_log(rng, 1, min(T, 200)), T=T, past=rng.choice([0, _log(rng, 1, 2000)]),
                    page=rng.choice([1, 16, 24, 64, 100, 256]), Hq=g * Hk, Hk=Hk, D=D, rot=rot,
                    off=rng.choice([0, D - rot]), inter=rng.random() < 0.5, dtype=dtype,
                    wtype=rng.choice([dtype, "fp32"]))
    block = rng.choice([1, 2, 4, 8, 16, 32, 64])
    window = rng.choice([0, _log(rng, 1, 256)])
    if kind == "paged":
        N, nq = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 5])
        W = _log(rng, 17, min(131072, 64 * 32768 * 8 // (N * Hk)))
        while 4 * block > W and block > 1:  # the shortest sequence has a complete block
            block //= 2
        slots = 64 * (2048 + 128) * 8 // (N * Hk)
        K = _log(rng, 1, max(1, min(2048, W // block + 1, slots // block)))
        return dict(op="paged", N=N, nq=nq, W=W, page=rng.choice([1, 16, 24, 64, 100, 256]), Hq=g * Hk, Hk=Hk, D=D, K=K,
                    block=block, window=window, dtype=dtype)
    train = kind == "sparse_train"
    T = _log(rng, 30, 8192 if train else 16384)
    most = (8192 * 256 if train else 16384 * 512) * 64 * 128  # list entries x heads x head size
    slots = max(1, most // (2 * T * g * Hk * D))
    rate = 0
    if rng.random() < 0.4:
        block, window, rate = 1, 0, rng.choice([1, 4, 8])
    docs = _log(rng, 1, max(1, T // 20))
    while block * docs * 4 > T and block > 1:  # most documents have a complete block
        block //= 2
    K = _log(rng, 1, max(1, min(1024, T // block, slots // block)))
    return dict(op="sparse", T=T, docs=docs, Hq=g * Hk, Hk=Hk, D=D, K=K, block=block,
                window=min(window, slots), rate=rate, prefix=rng.choice([0, _log(rng, 1, 1000)]) if not rate else 0,
                ragged=rng.random() < 0.5, dtype=dtype, train=train)


# ----------------------------------------------------------------------------- sizes of a case (host)
def _lengths(case):
    """Query and key lengths of the packed sequences: the case's own, so that every seed has the same shapes."""
    T, n = case["T"], case["docs"]
    rng = np.random.default_rng(T * 7919 + n)
    cuts = np.sort(rng.integers(1, T, n - 1)) if n > 1 else np.array([], dtype=np.int64)
    if case["ragged"] and n > 4:
        cuts[1] = cuts[0]          # an empty sequence
        cuts[3] = cuts[2] + 1      # a single token
        cuts = np.sort(np.minimum(cuts, T))
    lq = np.diff(np.concatenate([[0], cuts, [T]])).astype(np.int64)
    if case["rate"]:
        return [int(x) for x in lq], [int(x) // case["rate"] for x in lq]
    lk = lq.copy()
    if case["prefix"]:             # keys of earlier tokens in front of some sequences
        lk = lk + rng.integers(0, case["prefix"] + 1, n) * rng.integers(0, 2, n)
    if case["ragged"]:
        short = rng.integers(0, 6, n) == 0   # fewer keys than queries: the first rows see nothing
        lk = np.where(short, lk // 2, lk)
    return [int(x) for x in lq], [int(x) for x in lk]


def _paged_lengths(case):
    rng = np.random.default_rng(case["N"] * 104729 + case["W"])
    W = case["W"]
    length = rng.integers(max(1, W // 4), W + 1, case["N"])
    length[0] = W
    return [int(x) for x in length]


def _append_lengths(case):
    """Tokens to append and tokens cached before, of each sequence."""
    rng = np.random.default_rng(case["T"] * 31 + case["N"])
    T, n = case["T"], case["N"]
    if n == T:
        new = np.ones(n, dtype=np.int64)
    else:
        cuts = np.sort(rng.integers(0, T + 1, n - 1)) if n > 1 else np.array([], dtype=np.int64)
        new = np.diff(np.concatenate([[0], cuts, [T]])).astype(np.int64)
    past = rng.integers(case["past"] // 2, case["past"] + 1, n)
    return [int(x) for x in new], [int(x) for x in past]


def _rows(case):
    """Per query row: position in its sequence (the last query stands at the last key), keys of the sequence, blocks
    that may be listed (the complete ones; entries: those whose tokens are all there)."""
    if case["op"] == "paged":
        lk = _paged_lengths(case)
        lq = [case["nq"]] * case["N"]
    else:
        lq, lk = _lengths(case)
    pos = np.concatenate([np.arange(a) + (0 if case.get("rate") else b - a) for a, b in zip(lq, lk)])
    keys = np.repeat(np.array(lk, dtype=np.int64), np.array(lq))
    unit = case.get("rate") or case["block"]
    last = np.minimum((pos + 1) // unit, keys if case.get("rate") else keys // unit)
    return lq, lk, pos, keys, np.maximum(0, last)


def _seen(case):
    """Keys that each row sees (at most: a listed block may lie in the window)."""
    _, _, pos, keys, avail = _rows(case)
    n = np.minimum(avail, case["K"]) * case["block"]
    if not case.get("rate"):
        n = np.minimum(n + np.minimum(np.maximum(pos + 1, 0), case["window"]), np.maximum(pos + 1, 0))
    return n


# ----------------------------------------------------------------------------- inputs
def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def _freqs(rot):
    """Turns per position of each pair as 64-bit fixed-point fractions: the table that the library's calls take."""
    turns = [int(round(THETA ** (-i / rot) / (2 * math.pi) * 2.0 ** 64)) for i in range(0, rot, 2)]
    return torch.tensor(np.array(turns, dtype=np.uint64).view(np.int64), device="cuda")


def _select(avail, K, gen):
    """Lists as the indexer writes them: of the `avail` blocks of each row the K with the largest scores, ascending,
    -1 behind.  Some blocks are in favour with all rows, and recent ones with each."""
    rows, n = len(avail), int(max(avail, default=0))
    idx = torch.full((rows, K), -1, dtype=torch.int32, device="cuda")
    if n == 0:
        return idx
    a = torch.tensor(avail, device="cuda")
    j = torch.arange(n, device="cuda")
    favour = torch.randn(n, generator=gen, device="cuda")
    step = max(1, (1 << 27) // n)
    for r in range(0, rows, step):
        last = a[r:r + step, None]
        s = favour + torch.randn(last.shape[0], n, generator=gen, device="cuda")
        s += 3 * torch.exp((j - last).clamp_(max=0) / 16)
        s.masked_fill_(j >= last, -math.inf)
        top, i = torch.topk(s, min(K, n))
        i = torch.where(top == -math.inf, n, i).sort(-1).values
        idx[r:r + step, :i.shape[1]] = torch.where(i == n, -1, i).int()
    return idx


def _pages(case, lengths, extra):
    """Page table [N, width] of a shuffled pool and the pool's size; pages past a sequence's end are -1."""
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    pool = sum(need) + extra
    order = np.random.default_rng(pool).permutation(pool)
    table = np.full((case["N"], max(need) + 1), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return torch.tensor(table, device="cuda"), pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    st = dict(case)
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if case["op"] == "append":
        new, past = _append_lengths(case)
        T = case["T"]
        # queries, keys and values as they leave the projection: views of one wider row, of uneven size per head
        qkv = randn(T, Hq + 2 * Hk, D) * torch.exp(0.5 * randn(1, Hq + 2 * Hk, 1, dtype=torch.float32)).to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        wt = DTYPES[case["wtype"]]
        st["qw"] = (1 + 0.2 * randn(D, dtype=torch.float32)).to(wt)
        st["kw"] = (1 + 0.2 * randn(D, dtype=torch.float32)).to(wt)
        st["cu_q"] = _cu(new)
        st["k_len"] = torch.tensor([a + b for a, b in zip(new, past)], dtype=torch.int32, device="cuda")
        st["pos"] = torch.tensor(np.concatenate([np.arange(a) + b for a, b in zip(new, past)]), device="cuda")
        st["table"], pool = _pages(case, [a + b for a, b in zip(new, past)], 3)
        st["k_pages"], st["v_pages"] = randn(pool, case["page"], Hk, D), randn(pool, case["page"], Hk, D)
        st["inv"] = THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        st["freqs"] = _freqs(case["rot"])
        return st
    st["scale"] = 1.0 / math.sqrt(D)
    lq, lk, _, _, avail = _rows(case)
    st["idx"] = _select(avail, case["K"], gen)
    st["lq"], st["lk"] = lq, lk
    st["cu_q"] = _cu(lq)
    st["q"] = randn(sum(lq), Hq, D)
    if case["op"] == "paged":
        st["k_len"] = torch.tensor(lk, dtype=torch.int32, device="cuda")
        st["table"], pool = _pages(case, lk, 3)
        st["k_pages"], st["v_pages"] = randn(pool, case["page"], Hk, D), randn(pool, case["page"], Hk, D)
        return st
    kv = randn(sum(lk), 2 * Hk, D)
    st["k"], st["v"] = kv[:, :Hk], kv[:, Hk:]
    st["cu_k"] = _cu(lk)
    if case["train"]:
        st["dout"] = randn(sum(lq), Hq, D)
    return st


# ----------------------------------------------------------------------------- plain forms
def _turned(x, w, st):
    """Norm and rotation of x [T,H,D] in 32 bits, the angles in 64 (far positions)."""
    a = st["pos"].to(torch.float64)[:, None] * st["inv"][None, :]
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    x32 = x.float()
    y = x32 * torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS) * w.float()
    z = y[..., st["off"]:st["off"] + st["rot"]]
    u, v = (z[..., 0::2], z[..., 1::2]) if st["inter"] else (z[..., :st["rot"] // 2], z[..., st["rot"] // 2:])
    nu, nv = u * cos - v * sin, u * sin + v * cos
    u.copy_(nu)
    v.copy_(nv)
    return y.to(x.dtype)


def _append_plain(st):
    T = st["T"]
    rows = torch.arange(T, device="cuda")
    seq = torch.searchsorted(st["cu_q"][1:].long(), rows, right=True)
    at = st["k_len"].long()[seq] - (st["cu_q"].long()[seq + 1] - rows)
    page = st["table"].long()[seq, at // st["page"]]
    st["k_pages"][page, at % st["page"]] = _turned(st["k"], st["kw"], st)
    st["v_pages"][page, at % st["page"]] = st["v"]
    return dict(q_out=_turned(st["q"], st["qw"], st), k_pages=st["k_pages"], v_pages=st["v_pages"])


def _slots(st, rows, seq):
    """Keys of the given rows, counted in their sequence: [R, window + K * block], and which of them count."""
    cu_q, K, block, window = st["cu_q"].long(), st["K"], st["block"], st["window"]
    lk = (st["k_len"].long() if "k_len" in st else st["cu_k"].long().diff())[seq]
    causal = not st.get("rate")
    pos = rows - cu_q[seq] + lk - cu_q.diff()[seq] if causal else lk - 1
    near = pos[:, None] - torch.arange(window, device="cuda")
    b = st["idx"][rows].long()
    far = (b[:, :, None] * block + torch.arange(block, device="cuda")).flatten(1)
    ok_far = (b >= 0).repeat_interleave(block, 1) & (far < lk[:, None]) & (far <= (pos - window)[:, None])
    keys, ok = torch.cat([near, far], 1), torch.cat([near >= 0, ok_far], 1)
    return torch.where(ok, keys, 0), ok


def _attend_plain(st):
    """Rows in blocks: the gathered keys of all rows would not fit the card."""
    q, scale = st["q"], st["scale"]
    T, Hq, D = q.shape
    Hk, g = st["Hk"], st["Hq"] // st["Hk"]
    paged = st["op"] == "paged"
    train = st.get("train", False)
    k, v = (st["k_pages"].flatten(0, 1), st["v_pages"].flatten(0, 1)) if paged else (st["k"], st["v"])
    cu_q = st["cu_q"].long()
    out = torch.zeros_like(q)
    lse = torch.full((T, Hq), -math.inf, device="cuda")
    if train:
        dq = torch.zeros_like(q)
        dk, dv = torch.zeros(k.shape, device="cuda"), torch.zeros(v.shape, device="cuda")
    width = st["window"] + st["K"] * st["block"]
    step = max(1, min(T, (1 << 28) // (width * max(Hk * D, Hq))))
    for r in range(0, T, step):
        rows = torch.arange(r, min(T, r + step), device="cuda")
        seq = torch.searchsorted(cu_q[1:], rows, right=True)
        keys, ok = _slots(st, rows, seq)
        if paged:
            at = st["table"].long()[seq[:, None], keys // st["page"]].clamp(min=0) * st["page"] + keys % st["page"]
        else:
            at = (st["cu_k"].long()[seq][:, None] + keys).clamp(max=max(0, k.shape[0] - 1))
        if k.shape[0] == 0:
            break
        R = len(rows)
        kk = k[at].permute(0, 2, 1, 3).float()   # [R, Hk, slots, D]
        vv = v[at].permute(0, 2, 1, 3).float()
        q32 = q[rows].float().reshape(R, Hk, g, D)
        s = (q32 @ kk.transpose(-1, -2)) * scale
        s.masked_fill_(~ok[:, None, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
        l = p.sum(-1, keepdim=True)
        p = p / torch.where(l == 0, 1.0, l)
        o = p @ vv
        out[rows] = o.reshape(R, Hq, D).to(q.dtype)
        lse[rows] = (m + torch.log(l)).reshape(R, Hq)
        if train:
            do = st["dout"][rows].float().reshape(R, Hk, g, D)
            ds = p * (do @ vv.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)) * scale
            dq[rows] = (ds @ kk).reshape(R, Hq, D).to(q.dtype)
            dk.index_add_(0, at.flatten(), (ds.transpose(-1, -2) @ q32).permute(0, 2, 1, 3).flatten(0, 1))
            dv.index_add_(0, at.flatten(), (p.transpose(-1, -2) @ do).permute(0, 2, 1, 3).flatten(0, 1))
    if train:
        return dict(out=out, lse=lse, dq=dq, dk=dk.to(k.dtype), dv=dv.to(v.dtype))
    return dict(out=out, lse=lse)


# ----------------------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    return _append_plain(st) if st["op"] == "append" else _attend_plain(st)


def _run_own(st):
    import sparse_attention_indexer_csa_gb300 as csa

    if st["op"] == "append":
        q_out = csa.norm_rope_append(st["q"], st["k"], st["v"], st["qw"], st["kw"], st["pos"], st["freqs"], st["cu_q"],
                                     st["k_len"], st["k_pages"], st["v_pages"], st["table"], eps=EPS,
                                     rot_offset=st["off"], interleaved=st["inter"])
        return dict(q_out=q_out, k_pages=st["k_pages"], v_pages=st["v_pages"])
    if st["op"] == "paged":
        out, lse = csa.sparse_attn_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["idx"], st["cu_q"],
                                         st["k_len"], st["scale"], block=st["block"], window=st["window"])
        return dict(out=out, lse=lse)
    kw = dict(block=st["block"], window=st["window"], causal=not st["rate"])
    out, lse = csa.sparse_attn_forward(st["q"], st["k"], st["v"], st["idx"], st["cu_q"], st["cu_k"], st["scale"], **kw)
    if not st["train"]:
        return dict(out=out, lse=lse)
    dq, dk, dv = csa.sparse_attn_backward(st["dout"], st["q"], st["k"], st["v"], out, lse, st["idx"], st["cu_q"],
                                          st["cu_k"], st["scale"], **kw)
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        we = 4 if case["wtype"] == "fp32" else 2
        return dict(bytes=2 * T * (Hq + 2 * Hk) * D * e + 12 * T + 2 * D * we + case["rot"] * 4 + 8 * case["N"],
                    flops=8 * T * (Hq + Hk) * D)
    seen = _seen(case)
    pairs, rows = int(seen.sum()) * Hq, len(seen)
    lists = int(np.minimum(_rows(case)[4], case["K"]).sum()) * 4
    nq, small = rows * Hq * D * e, rows * Hq * 4 + lists + 8 * case.get("N", 1)
    if case["op"] == "paged":  # each row's keys; the rows of a sequence may share some, as the lists come
        lq, lk = [case["nq"]] * case["N"], _paged_lengths(case)
        per = seen.reshape(case["N"], case["nq"]).max(1)
        return dict(bytes=2 * int(per.sum()) * Hk * D * e + 2 * nq + small, flops=4 * D * pairs)
    nk = sum(_lengths(case)[1]) * Hk * D * e
    if case["train"]:
        return dict(bytes=4 * nq + 4 * nk + small, flops=14 * D * pairs)
    return dict(bytes=2 * nq + 2 * nk + small, flops=4 * D * pairs)


# ----------------------------------------------------------------------------- the definition in 64 bits
def _exact_append(st):
    """Norm and rotation as products of complex numbers; tokens put into their pages one sequence after the other."""
    pos, rot, off, page = st["pos"].double(), st["rot"], st["off"], st["page"]
    expo = torch.arange(rot // 2, dtype=torch.float64, device="cuda") * (-2.0 / rot)
    unit = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                       pos.unsqueeze(1) * torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"), expo))

    def turned(x, w):
        x = x.double()
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
        body = y[..., off:off + rot]
        pairs = body.unflatten(-1, (rot // 2, 2)) if st["inter"] else body.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        flat = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit[:, None, :])
        flat = flat.flatten(-2) if st["inter"] else flat.transpose(-1, -2).flatten(-2)
        return torch.cat([y[..., :off], flat, y[..., off + rot:]], -1)

    q_out, k_new, v_new = turned(st["q"], st["qw"]), turned(st["k"], st["kw"]), st["v"].double()
    caches = [st["k_pages"].double().flatten(0, 1), st["v_pages"].double().flatten(0, 1)]
    new, past = _append_lengths(st)
    table, a = st["table"].cpu().numpy(), 0
    for i, (n, p) in enumerate(zip(new, past)):
        at = np.arange(p, p + n)
        rows = torch.tensor(table[i][at // page].astype(np.int64) * page + at % page, device="cuda")
        for cache, x in zip(caches, (k_new, v_new)):
            cache[rows] = x[a:a + n]
        a += n
    shape = st["k_pages"].shape
    return dict(q_out=q_out, k_pages=caches[0].reshape(shape), v_pages=caches[1].reshape(shape))


def _mask(st, idx, pos, lk):
    """[rows, lk]: the keys of one sequence that each row sees."""
    block, window = st["block"], st["window"]
    nb = -(-lk // block)
    hit = torch.zeros(len(pos), nb + 1, dtype=torch.bool, device="cuda")
    hit.scatter_(1, torch.where(idx < 0, nb, idx).long(), True)
    see = hit[:, :nb].repeat_interleave(block, 1)[:, :lk]
    if st.get("rate"):
        return see
    j = torch.arange(lk, device="cuda")[None]
    return (see | (j > pos[:, None] - window)) & (j <= pos[:, None])


def _exact_attend(st):
    Hq, Hk, D, scale = st["Hq"], st["Hk"], st["D"], st["scale"]
    g, train, T = Hq // Hk, st.get("train", False), st["q"].shape[0]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    if train:
        grads = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in (st["q"], st["k"], st["v"])]
    a = c = 0
    for i, (lq, lk) in enumerate(zip(st["lq"], st["lk"])):
        if lk and lq:
            if st["op"] == "paged":
                at = torch.arange(lk, device="cuda")
                at = st["table"][i].long()[at // st["page"]] * st["page"] + at % st["page"]
                keys, values = st["k_pages"].flatten(0, 1)[at], st["v_pages"].flatten(0, 1)[at]
            else:
                keys, values = st["k"][c:c + lk], st["v"][c:c + lk]
            step = max(1, (1 << 26) // (g * lk))
            for r in range(0, lq, step):
                n = min(step, lq - r)
                rows = slice(a + r, a + r + n)
                see = _mask(st, st["idx"][rows], torch.arange(r, r + n, device="cuda") + lk - lq, lk)
                some = see.any(1)
                for h in range(Hk):
                    heads = slice(h * g, (h + 1) * g)
                    leaves = [st["q"][rows, heads].double(), keys[:, h].double(), values[:, h].double()]
                    if train:
                        leaves = [t.requires_grad_(True) for t in leaves]
                    s = torch.matmul(leaves[0], leaves[1].T) * scale
                    s = s.masked_fill(~see[:, None] & some[:, None, None], -math.inf)
                    w = torch.softmax(s, -1) * some[:, None, None]
                    o = torch.matmul(w, leaves[2])
                    out[rows, heads] = o.detach()
                    l = torch.logsumexp(s.detach(), -1)
                    lse[rows, heads] = torch.where(some[:, None], l, -math.inf)
                    if train:
                        d = torch.autograd.grad(o, leaves, st["dout"][rows, heads].double())
                        grads[0][rows, heads] += d[0]
                        grads[1][c:c + lk, h] += d[1]
                        grads[2][c:c + lk, h] += d[2]
        a, c = a + lq, c + lk
    if train:
        return dict(out=out, lse=lse, dq=grads[0], dk=grads[1], dv=grads[2])
    return dict(out=out, lse=lse)


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attend(st)
