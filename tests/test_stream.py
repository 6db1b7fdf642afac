"""The stream that a call goes to where none is given: the current one, with or without torch's function
for its handle."""
import types

import pytest
import torch

T = pytest.importorskip("tree_masked_gated_amd")


@pytest.mark.parametrize("raw", [None, lambda device: {3: 77}[device]])
def test_handle_without_the_private_function(monkeypatch, raw):
    monkeypatch.setattr(T, "_raw_stream", raw)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert T._stream(None) == 77
    assert T._stream(5) == 5 and T._stream(types.SimpleNamespace(cuda_stream=9)) == 9


@pytest.mark.gpu
def test_handle_is_the_current_stream():
    side = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), side, torch.cuda.default_stream()):
        with torch.cuda.stream(s):
            assert T._stream(None) == torch.cuda.current_stream().cuda_stream == s.cuda_stream
