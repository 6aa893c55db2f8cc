"""The binding's handling of devices and streams."""
import pytest
import torch

import sparse_attention_indexer_csa_gb300 as csa
from sparse_attention_indexer_csa_gb300 import attn


def test_a_refused_stream_leaves_the_current_device_alone(monkeypatch):
    entered = []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *_):
            entered.remove(self.device)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(attn, "_current_stream", lambda device: 0)
    other = torch.device("cuda", 1)
    with pytest.raises(TypeError):
        attn._Call(object(), other)
    assert not entered
    call = attn._Call(None, other)  # and a call's own lasts until it is done
    assert entered == [other]
    call.done()
    assert not entered


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["norm_rope", "norm_rope_backward", "attn_forward", "attn_backward"])
def test_inputs_may_be_dropped_while_a_side_stream_still_reads_them(op):
    """The memory of inputs that nobody holds any more goes to other work only after the call's stream is through."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    T, H, D = 1111, 4, 64
    keep = [r(T, H, D) for _ in range(4)]
    w, pos, fr = torch.ones(D, device="cuda"), torch.arange(T, device="cuda"), csa.rope_freqs(D)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out, lse = csa.attn_forward(*keep[:3], cu, cu, 0.125)

    def call(t, stream=None):
        if op == "norm_rope":
            return csa.norm_rope(t[0], t[1], w, w, pos, fr, stream=stream)
        if op == "norm_rope_backward":
            return csa.norm_rope_backward(*t, w, w, pos, fr, stream=stream)
        if op == "attn_forward":
            return csa.attn_forward(*t[:3], cu, cu, 0.125, stream=stream)
        return csa.attn_backward(t[3], *t[:3], out, lse, cu, cu, 0.125, stream=stream)

    want = call(keep)
    torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")  # its kernel is loaded before the race
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    copies = [t.clone() for t in keep]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # a tenth of a second
    got = call(copies, stream=side)
    del copies
    others = [torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(16)]  # other work
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert len(others) == 16 and csa.device_status() == csa.CSA_OK
