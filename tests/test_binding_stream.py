"""The stream a call goes to when none is given, on the host: the current one's handle, whether or not torch has its private
name for it."""
import types

import torch

from bit_kv_cache_13_gb300 import _lib


def test_current_stream_with_and_without_the_private_name(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=1000 + dev))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 2000 + dev, raising=False)
    assert _lib._stream(None) == 2001
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert _lib._stream(None) == 1001


def test_given_streams():
    assert _lib._stream(types.SimpleNamespace(cuda_stream=7)) == 7 and _lib._stream(5) == 5
