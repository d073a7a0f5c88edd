"""The stream that a call of the binding runs on: the current one of the context's device."""

import importlib.util
import sys
import types

import pytest
import torch

from rank_markov_draft_gb300 import binding


def test_current_stream_without_the_private_call(monkeypatch):
    """A torch that does not have the call for the bare handle is asked for the stream."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=100 + d))
    spec = importlib.util.spec_from_file_location("rank_markov_draft_gb300.binding_again", binding.__file__)
    again = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, spec.name, again)
    spec.loader.exec_module(again)
    assert again._stream(None, 3) == 103
    assert again._stream(None, torch.device("cuda", 2)) == 102
    assert again._stream(77, 3) == 77


@pytest.mark.gpu
def test_current_stream_is_torchs():
    side = torch.cuda.Stream()
    for stream in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(stream):
            assert binding._stream(None, 0) == stream.cuda_stream
            assert binding._stream(None, torch.device("cuda")) == stream.cuda_stream
        assert binding._stream(stream, 0) == stream.cuda_stream
