"""The stream that the binding's calls take when none is given."""
from types import SimpleNamespace

import pytest
import torch


def test_current_stream_without_torchs_own_look_up(hd, monkeypatch):
    """That look-up is no public function of torch: without it the binding takes the public one."""
    asked = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: asked.append(device) or SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(hd, "_raw_stream", hd._stream_lookup(SimpleNamespace()))
    assert hd._stream(None) == 77 and asked == [3]
    monkeypatch.setattr(hd, "_raw_stream", hd._stream_lookup(SimpleNamespace(_cuda_getCurrentRawStream=lambda device: 100 + device)))
    assert hd._stream(None) == 103
    assert hd._stream(5) == 5


@pytest.mark.gpu
def test_current_stream_is_the_same_either_way(hd):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    s = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), s):
        with torch.cuda.stream(stream):
            assert hd._stream(None) == hd._stream_lookup(object())(torch.cuda.current_device()) == stream.cuda_stream
