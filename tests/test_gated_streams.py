"""The binding finds the current device and stream through torch's public calls where the short ways are missing."""
import importlib.util

import pytest
import torch

L = pytest.importorskip("causal_linear_attention_attn_gb300.linattn")


def without_short_ways(monkeypatch):
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("linattn_by_public_calls", L.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_public_calls(monkeypatch):
    m = without_short_ways(monkeypatch)
    assert m._device_index is torch.cuda.current_device

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: Stream)
    assert m._stream_handle(0) == 77


@pytest.mark.gpu
def test_the_current_stream_by_either_way(cuda_lib):
    side = torch.cuda.Stream()
    for s in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(s):
            assert cuda_lib._on(torch.device("cuda", 0), None) == (s.cuda_stream, None)
            assert cuda_lib._device_index() == torch.cuda.current_device() == 0
            assert cuda_lib._stream_handle(0) == torch.cuda.current_stream(0).cuda_stream
