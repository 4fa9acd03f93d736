"""The binding's stream handles (no GPU): the current stream with and without PyTorch's shortcut for it."""
import importlib

import torch

import weight_only_int4_linear_b200 as w4


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_current_stream_without_the_shortcut(monkeypatch):
    """A PyTorch without the shortcut takes the public way; every entry point resolves its stream there."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: _Stream(1000 + index))
    spec = importlib.util.spec_from_file_location("binding_without_shortcut", w4.__file__)
    other = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(other)
    assert other._stream(None) == 1003
    assert other._stream(77) == 77


def test_current_stream_by_the_shortcut(monkeypatch):
    monkeypatch.setattr(w4, "_raw_stream", lambda index: 2000 + index)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 5)
    assert w4._stream(None) == 2005
