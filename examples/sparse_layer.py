"""One attention layer that reads only what its indexer selects, from training to serving.

Prompt: the queries and keys of the projections (views, no copies) are
normalised and rotated, the indexer selects compressed entries for every row of
every document, and attention runs over the tokens that the selected entries
stand for and the last WINDOW ones.  A loss on its output goes back to the
projections' weights.  Serving: the tokens of each document but the last go into
a paged cache, in two chunks; then a step appends the last token, selects with
its query and attends over the pages.

    python examples/sparse_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_csa_gb300 as csa  # noqa: E402

HQ, HK, D, ROT = 16, 2, 128, 64  # attention heads, head size, rotated values (the last ones of a head)
HI, RATE, TOP_K, WINDOW = 64, 4, 24, 16  # indexer heads, tokens of an entry, entries kept per row, last tokens read anyway
PAGE = 16  # tokens of a page of the cache
WIDTH = 256  # of the hidden states
THETA, EPS, SCALE = 10000.0, 1e-6, D ** -0.5
TURN = dict(eps=EPS, rot_offset=D - ROT)


def make_weights(seed=0, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=gen) * s[0] ** -0.5).bfloat16().to(device)  # noqa: E731
    one = lambda: (1 + 0.1 * torch.randn(D, generator=gen)).bfloat16().to(device)  # noqa: E731
    return dict(qkv=r(WIDTH, (HQ + 2 * HK) * D), q_norm=one(), k_norm=one(), index_q=r(WIDTH, HI * D),
                index_k=r(WIDTH, D), index_w=r(WIDTH, HI), iq_norm=one(), ik_norm=one(),
                freqs=csa.rope_freqs(ROT, THETA, device=device))


def cumulative(lengths, device):
    return torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=device)


def heads(x, w):
    """Queries, keys and values of hidden states x [T,WIDTH]: views of one product."""
    y = (x @ w["qkv"]).view(-1, HQ + 2 * HK, D)
    return y[:, :HQ], y[:, HQ:HQ + HK], y[:, HQ + HK:]


def index_queries(x, w, positions):
    q, _ = csa.norm_rope((x @ w["index_q"]).view(-1, HI, D), None, w["iq_norm"], None, positions, w["freqs"], **TURN)
    return q, x @ w["index_w"]


def index_entries(x, w):
    """One document's compressed entries [W,D]: the means of RATE tokens each, at the position of the first."""
    n = x.shape[0] // RATE
    at = torch.arange(0, n * RATE, RATE, device=x.device)
    pooled = x[:n * RATE].view(n, RATE, WIDTH).float().mean(1).bfloat16()
    k, _ = csa.norm_rope((pooled @ w["index_k"]).view(n, 1, D), None, w["ik_norm"], None, at, w["freqs"], **TURN)
    return k.view(n, D)


def select(x, w, lengths, positions):
    """idx [T,TOP_K]: for each row the entries it keeps, numbered within its document."""
    q, iw = index_queries(x, w, positions)
    idx = torch.full((x.shape[0], TOP_K), -1, dtype=torch.int32, device=x.device)
    a = 0
    for n in lengths:
        if n >= RATE:
            k = index_entries(x[a:a + n], w)
            idx[a:a + n] = csa.index_fused(q[None, a:a + n], k[None], iw[None, a:a + n].contiguous(), SCALE, RATE, TOP_K,
                                           q_layout=csa.CSA_Q_SEQ_MAJOR)[0]
        a += n
    return idx


def prompt(x, w, lengths):
    """Forward of packed documents; what the backward needs is returned."""
    dev = x.device
    cu = cumulative(lengths, dev)
    positions = torch.cat([torch.arange(n, device=dev) for n in lengths])
    q0, k0, v = heads(x, w)
    q, k = csa.norm_rope(q0, k0, w["q_norm"], w["k_norm"], positions, w["freqs"], **TURN)
    idx = select(x, w, lengths, positions)
    out, lse = csa.sparse_attn_forward(q, k, v, idx, cu, cu, SCALE, block=RATE, window=WINDOW)
    return dict(x=x, cu=cu, positions=positions, q0=q0, k0=k0, q=q, k=k, v=v, idx=idx, out=out, lse=lse)


def prompt_backward(s, w, dout):
    """Gradients of the weights for the cotangent dout of the output."""
    dq, dk, dv = csa.sparse_attn_backward(dout, s["q"], s["k"], s["v"], s["out"], s["lse"], s["idx"], s["cu"], s["cu"],
                                          SCALE, block=RATE, window=WINDOW)
    dq0, dk0, d_qn, d_kn = csa.norm_rope_backward(dq, dk, s["q0"], s["k0"], w["q_norm"], w["k_norm"], s["positions"],
                                                  w["freqs"], **TURN)
    dy = torch.cat([dq0, dk0, dv], dim=1).view(s["x"].shape[0], -1)
    return dict(qkv=s["x"].t() @ dy, q_norm=d_qn, k_norm=d_kn)


class Cache:
    """Pages of keys and values for sequences of up to `most` tokens, dealt out in a shuffled order."""

    def __init__(self, n, most, device="cuda", seed=0):
        width = -(-most // PAGE)
        order = torch.randperm(n * width, generator=torch.Generator().manual_seed(seed))
        self.table = order.view(n, width).int().to(device)
        self.k, self.v = (torch.full((n * width, PAGE, HK, D), float("nan"), dtype=torch.bfloat16, device=device)
                          for _ in range(2))
        self.lens = torch.zeros(n, dtype=torch.int32, device=device)

    def append(self, x, w, new):
        """Tokens x [sum(new),WIDTH] behind the sequences -> their queries, normalised and rotated, and cu_q."""
        cu = cumulative(new, x.device)
        before = self.lens.long()
        self.lens = self.lens + cu.diff()
        positions = torch.cat([torch.arange(n, device=x.device) + before[i] for i, n in enumerate(new)])
        q0, k0, v = heads(x, w)
        q = csa.norm_rope_append(q0, k0, v, w["q_norm"], w["k_norm"], positions, w["freqs"], cu, self.lens, self.k, self.v,
                                 self.table, **TURN)
        return q, cu, positions


def step(x, w, cache, entries):
    """One token x [N,WIDTH] of each sequence: appended, then attending over the cache.  entries [N,W,D]: the indexer's,
    of the complete groups of RATE tokens, the one among them that this token completes."""
    N = x.shape[0]
    q, cu, positions = cache.append(x, w, [1] * N)
    iq, iw = index_queries(x, w, positions)
    idx = csa.index_fused(iq.view(N, 1, HI, D), entries, iw.view(N, 1, HI), SCALE, RATE, TOP_K, q_start=positions,
                          q_layout=csa.CSA_Q_SEQ_MAJOR).view(N, TOP_K)
    out, _ = csa.sparse_attn_paged(q, cache.k, cache.v, cache.table, idx, cu, cache.lens, SCALE, block=RATE,
                                   window=WINDOW)
    return out, idx, q


def run(lengths=(300, 9, 129, 514), seed=0):
    w = make_weights(seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(sum(lengths), WIDTH, generator=gen).bfloat16().cuda()
    s = prompt(x, w, lengths)
    target = torch.randn(s["out"].shape, generator=gen).cuda()
    diff = s["out"].float() - target
    loss = 0.5 * diff.square().mean()
    grads = prompt_backward(s, w, (diff / diff.numel() * 2 ** 16).bfloat16())  # scaled, as mixed precision does
    # The same documents served: all tokens but the last in two chunks, then a step.
    docs = list(x.split(list(lengths)))
    cache = Cache(len(docs), max(lengths))
    for part in ([d[:(len(d) - 1) // 2] for d in docs], [d[(len(d) - 1) // 2:len(d) - 1] for d in docs]):
        cache.append(torch.cat(part), w, [len(p) for p in part])
    entries = torch.zeros(len(docs), max(1, max(lengths) // RATE), D, dtype=torch.bfloat16, device="cuda")
    for i, d in enumerate(docs):
        if len(d) >= RATE:
            entries[i, :len(d) // RATE] = index_entries(d, w)
    last = s["cu"][1:].long() - 1
    again, idx, q = step(x[last], w, cache, entries)
    torch.cuda.synchronize()
    if csa.device_status() != csa.CSA_OK:
        raise RuntimeError("device status word reports an error")
    return dict(s, loss=loss, grads=grads, step=again, step_idx=idx, step_q=q, last=last, weights=w, cache=cache, target=target)


if __name__ == "__main__":
    r = run()
    print(f"loss {r['loss'].item():.4f}; "
          f"largest gradient of the projection {r['grads']['qkv'].abs().max().item() / 2 ** 16:.2e}; "
          f"entries kept by the last row {(r['idx'][-1] >= 0).sum().item()}; "
          f"step against prompt {(r['step'].float() - r['out'][r['last']].float()).abs().max().item():.2e}")
