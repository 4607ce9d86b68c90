"""The binding under a torch without the private lookups of the current device and stream."""
import importlib.util

import torch

import sparse_mixture_experts_argmax_b200 as swl


def test_public_lookups_stand_in_for_private_ones(monkeypatch):
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("swl_without_private_names", swl.__file__)
    other = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(other)

    class Stream:
        cuda_stream = 1234

    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: asked.append(d) or Stream())
    monkeypatch.setattr(other, "_current_device", lambda: 3)
    assert other._stream_handle(None) == 1234 and asked == [3]
    assert other._stream_handle(77) == 77
    assert other._on(torch.device("cuda", 3)) is other._HERE_ALREADY
