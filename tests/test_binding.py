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


@pytest.mark.gpu
def test_a_workspace_that_only_looks_large_is_refused():
    thin = torch.empty(16, dtype=torch.uint8, device="cuda").expand(1 << 20, 16)     # 16 bytes
    q, k = torch.zeros(1, 4, 64, device="cuda"), torch.zeros(16, 2, 64, device="cuda")
    b = L.Batch(torch.tensor([16], dtype=torch.int32, device="cuda"), 1, 16)
    x = torch.zeros(32, 4, device="cuda")
    t, i = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for f in (lambda: L.dense_attn(q, k, k, b, 1.0, workspace=thin),
              lambda: L.idx_page_update(t, i, i, i, 4, [x], workspace=thin),
              lambda: L.idx_page_compact(t, i, 4, [x], workspace=thin)):
        with pytest.raises(ValueError, match="workspace"):
            f()


@pytest.mark.gpu
@pytest.mark.parametrize("name,shape", [("q_pos", (5,)), ("kv_start", (2,)), ("page_table", (2, 4))])
def test_batch_arrays_shorter_than_the_batch_are_refused(name, shape):
    # three sequences of two rows
    q, k = torch.zeros(6, 4, 64, device="cuda"), torch.zeros(64, 2, 64, device="cuda")
    n_kv = torch.full((3,), 16, dtype=torch.int32, device="cuda")
    b = L.Batch(n_kv, 2, 16, page_size=4, **{name: torch.zeros(shape, dtype=torch.int32, device="cuda")})
    with pytest.raises(ValueError, match=name):
        L.dense_attn(q, k, k, b, 1.0)
    if name == "kv_start":      # not read beside a page table
        b.page_table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
        assert (L.dense_attn(q, k, k, b, 1.0) == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(window=4 - 2**32), dict(window=-2**31 - 1), dict(softcap=1e-60), dict(softcap=-1e-60)])
def test_options_that_change_on_their_way_to_32_bits_are_refused(kw):
    q, k = torch.zeros(1, 4, 64, device="cuda"), torch.zeros(16, 2, 64, device="cuda")
    b = L.Batch(torch.tensor([16], dtype=torch.int32, device="cuda"), 1, 16,
                q_pos=torch.tensor([15], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match=next(iter(kw))):
        L.dense_attn(q, k, k, b, 1.0, **kw)
