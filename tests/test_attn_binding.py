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
