"""The binding's own parts."""

import types

import pytest
import torch

import lightning_indexer_top_gb300 as L


def test_the_stream_of_a_device_without_the_raw_accessor(monkeypatch):
    asked = []

    def current_stream(device):
        asked.append(device)
        return types.SimpleNamespace(cuda_stream=1234)
    monkeypatch.setattr(L, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    dev = torch.device("cuda", 1)
    assert L._stream(dev) == 1234 and asked == [dev]


@pytest.mark.gpu
def test_both_ways_to_the_current_stream_agree(monkeypatch):
    dev = torch.empty(1, device="cuda").device
    other = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), other):
        with torch.cuda.stream(stream):
            here = L._stream(dev)
            with monkeypatch.context() as m:
                m.setattr(L, "_raw_stream", None)
                assert L._stream(dev) == here == stream.cuda_stream
