"""The current stream's handle where torch lacks either of the two functions
that give it directly: from the stream object."""
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M


class _Stream:
    cuda_stream = 1234


@pytest.mark.parametrize("missing", [["_raw_stream"], ["_raw_device"], ["_raw_stream", "_raw_device"]])
def test_without_the_direct_functions(monkeypatch, missing):
    for name in ("_raw_stream", "_raw_device"):
        monkeypatch.setattr(M, name, None if name in missing else lambda *a: pytest.fail("called"))
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: _Stream)
    assert M._stream().value == 1234


def test_a_given_stream_is_taken(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: pytest.fail("called"))
    assert M._stream(_Stream).value == 1234


@pytest.mark.gpu
def test_current_streams():
    torch.zeros(1, device="cuda")
    assert (M._stream().value or 0) == torch.cuda.current_stream().cuda_stream
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        assert M._stream().value == st.cuda_stream
