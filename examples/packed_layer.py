"""One attention layer with its indexer over packed documents, as a program would run it.

Prompt: the queries and keys of the projections (views, no copies) are
normalised and rotated, the indexer selects compressed entries for every
row, attention runs over the documents, and a loss on its output goes back
through attention, rotation and norm to the projections' weights.  Then the
keys and values are put into a cache, and every document is continued by one
token.

    python examples/packed_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_csa_gb300 as csa  # noqa: E402

HQ, HK, D, ROT = 16, 2, 128, 64  # attention heads, head size, rotated values (the last ones of a head)
HI, RATE, TOP_K = 64, 4, 48  # indexer heads, tokens per compressed entry, entries kept per row
WIDTH = 256  # of the hidden states
THETA, EPS, SCALE = 10000.0, 1e-6, D ** -0.5


def make_weights(seed=0, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=gen) * s[0] ** -0.5).bfloat16().to(device)  # noqa: E731
    one = lambda: (1 + 0.1 * torch.randn(D, generator=gen)).bfloat16().to(device)  # noqa: E731
    return dict(qkv=r(WIDTH, (HQ + 2 * HK) * D), q_norm=one(), k_norm=one(), index_q=r(WIDTH, HI * D),
                index_k=r(WIDTH, D), index_w=r(WIDTH, HI), iq_norm=one(), ik_norm=one(),
                freqs=csa.rope_freqs(ROT, THETA, device=device))


def heads(x, w):
    """Queries, keys and values of hidden states x [T,WIDTH]: views of one product."""
    y = (x @ w["qkv"]).view(-1, HQ + 2 * HK, D)
    return y[:, :HQ], y[:, HQ:HQ + HK], y[:, HQ + HK:]


def turn(q, k, w, positions):
    return csa.norm_rope(q, k, w["q_norm"], w["k_norm"], positions, w["freqs"], eps=EPS, rot_offset=D - ROT)


def select(x, w, lengths, positions):
    """The indexer on one row of packed documents: idx [1,T,TOP_K].  An entry stands for RATE tokens of the row."""
    T = x.shape[0]
    if T < RATE:  # no entry yet
        return torch.full((1, T, TOP_K), -1, dtype=torch.int32, device=x.device)
    doc = torch.repeat_interleave(torch.arange(len(lengths), device=x.device, dtype=torch.int32),
                                  torch.tensor(lengths, device=x.device))
    kw = dict(eps=EPS, rot_offset=D - ROT)
    q, _ = csa.norm_rope((x @ w["index_q"]).view(T, HI, D), None, w["iq_norm"], None, positions, w["freqs"], **kw)
    at = torch.arange(0, T // RATE * RATE, RATE, device=x.device)  # the first token of each entry
    pooled = x[:T // RATE * RATE].view(-1, RATE, WIDTH).float().mean(1).bfloat16()
    k, _ = csa.norm_rope((pooled @ w["index_k"]).view(-1, 1, D), None, w["ik_norm"], None, positions[at], w["freqs"],
                         **kw)
    return csa.index_fused(q.view(1, T, HI, D), k.view(1, -1, D), (x @ w["index_w"]).view(1, T, HI), SCALE, RATE, TOP_K,
                           q_seg=doc.view(1, -1), kv_seg=doc[at].view(1, -1), q_layout=csa.CSA_Q_SEQ_MAJOR)


def prompt(x, w, lengths):
    """Forward of packed documents; what the backward and the cache need is returned."""
    dev = x.device
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=dev)
    positions = torch.cat([torch.arange(n, device=dev) for n in lengths])
    q0, k0, v = heads(x, w)
    q, k = turn(q0, k0, w, positions)
    out, lse = csa.attn_forward(q, k, v, cu, cu, SCALE)
    return dict(x=x, cu=cu, positions=positions, q0=q0, k0=k0, q=q, k=k, v=v, out=out, lse=lse)


def prompt_backward(s, w, dout):
    """Gradients of the weights for the cotangent dout of the output."""
    dq, dk, dv = csa.attn_backward(dout, s["q"], s["k"], s["v"], s["out"], s["lse"], s["cu"], s["cu"], SCALE)
    dq0, dk0, d_qn, d_kn = csa.norm_rope_backward(dq, dk, s["q0"], s["k0"], w["q_norm"], w["k_norm"], s["positions"],
                                                  w["freqs"], eps=EPS, rot_offset=D - ROT)
    dy = torch.cat([dq0, dk0, dv], dim=1).view(s["x"].shape[0], -1)
    return dict(qkv=s["x"].t() @ dy, q_norm=d_qn, k_norm=d_kn)


def fill_cache(s, lengths, width):
    """Cache [N,width,HK,D] of the documents' keys and values."""
    k, v = (torch.zeros(len(lengths), width, HK, D, dtype=s["k"].dtype, device=s["k"].device) for _ in range(2))
    at = 0
    for i, n in enumerate(lengths):
        k[i, :n], v[i, :n] = s["k"][at:at + n], s["v"][at:at + n]
        at += n
    return k, v


def step(x, w, cache, lens):
    """One token x [N,WIDTH] behind each document; lens [N] int32 are the lengths before it."""
    kc, vc = cache
    N, width = kc.shape[:2]
    q0, k0, v = heads(x, w)
    q, k = turn(q0, k0, w, lens.long())
    rows = torch.arange(N, device=x.device)
    kc[rows, lens.long()], vc[rows, lens.long()] = k, v
    cu = torch.arange(N + 1, device=x.device, dtype=torch.int32)
    out, _ = csa.attn_forward(q, kc.view(-1, HK, D), vc.view(-1, HK, D), cu, cu * width, SCALE, k_len=lens + 1)
    return out


def run(lengths=(300, 1, 129, 514), seed=0):
    w = make_weights(seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(sum(lengths), WIDTH, generator=gen).bfloat16().cuda()
    s = prompt(x, w, lengths)
    idx = select(x, w, lengths, s["positions"])
    target = torch.randn(s["out"].shape, generator=gen).cuda()
    diff = s["out"].float() - target
    loss = 0.5 * diff.square().mean()
    grads = prompt_backward(s, w, (diff / diff.numel() * 2 ** 16).bfloat16())  # scaled, as mixed precision does
    # The last token of each document once more, as a step behind the tokens before it.
    last = s["cu"][1:].long() - 1
    lens = torch.tensor([n - 1 for n in lengths], dtype=torch.int32, device=x.device)
    cache = fill_cache(s, lengths, max(lengths) + 1)
    again = step(x[last], w, cache, lens)
    torch.cuda.synchronize()
    if csa.device_status() != csa.CSA_OK:
        raise RuntimeError("device status word reports an error")
    return dict(s, loss=loss, grads=grads, idx=idx, step=again, last=last, weights=w)


if __name__ == "__main__":
    r = run()
    print(f"loss {r['loss'].item():.4f}; "
          f"largest gradient of the projection {r['grads']['qkv'].abs().max().item() / 2 ** 16:.2e}; "
          f"entries kept by the last row {(r['idx'][0, -1] >= 0).sum().item()}; "
          f"step against prompt {(r['step'].float() - r['out'][r['last']].float()).abs().max().item():.2e}")
