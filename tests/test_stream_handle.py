"""The stream that the binding passes on: torch's current one, by either way to its handle."""
import types

import pytest
import torch

from reconstruction_lact_chunk_amd import binding as B


def test_without_the_short_way(monkeypatch):
    device = torch.device("cuda", 3)
    asked = []
    monkeypatch.setattr(B, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d: asked.append(d) or types.SimpleNamespace(cuda_stream=12345))
    assert B._stream(device) == 12345 and asked == [device]


def test_with_the_short_way(monkeypatch):
    monkeypatch.setattr(B, "_raw_stream", lambda index: 100 + index)
    assert B._stream(torch.device("cuda", 3)) == 103


@pytest.mark.gpu
def test_both_name_the_current_stream(monkeypatch):
    device = torch.device("cuda", 0)
    short = [B._stream(device)]
    with torch.cuda.stream(torch.cuda.Stream()):
        short.append(B._stream(device))
    monkeypatch.setattr(B, "_raw_stream", None)
    assert B._stream(device) == short[0] == torch.cuda.current_stream(device).cuda_stream != short[1]
