"""What stream a call goes to, without a GPU."""
import types

import torch

import kv_cache_compression_layer_b200 as kv


def test_current_stream_without_the_private_entry(monkeypatch):
    """The raw stream comes from torch's public API where the private entry is missing."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=4096))
    assert kv._stream(None) == 4096


def test_given_streams():
    assert kv._stream(0) == 0 and kv._stream(4096) == 4096
    assert kv._stream(types.SimpleNamespace(cuda_stream=77)) == 77
