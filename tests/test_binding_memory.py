"""Where the binding's allocations come from: the stream that the call runs on (with stand-ins for torch's
streams and allocator, on the CPU)."""

import contextlib
import re

import pytest
import torch

from rank_markov_draft_gb300 import binding


class Stream:
    def __init__(self, name):
        self.cuda_stream, self.name = 0, name


class Tensor:
    device = "cuda:0"

    def __init__(self, made_on, shape):
        self.made_on, self.shape, self.recorded = made_on, shape, []

    def record_stream(self, s):
        self.recorded.append(s.name)


@pytest.fixture
def streams(monkeypatch):
    """torch with a current stream that `with torch.cuda.stream(s)` changes, and tensors that remember it."""
    at = [Stream("callers")]

    @contextlib.contextmanager
    def stream(s):
        at.append(s)
        yield
        at.pop()

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(f"handle {handle}"))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: at[-1])
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Tensor(at[-1].name, shape))


def test_memory_is_the_calls_streams(streams):
    t = binding._empty(Stream("side"), (2, 3), torch.float32, "cuda:0")
    assert (t.made_on, t.shape, t.recorded) == ("side", (2, 3), ["callers"])
    t = binding._empty(1234, (2,), torch.float32, "cuda:0")
    assert (t.made_on, t.recorded) == ("handle 1234", ["callers"])
    t = binding._empty(None, (2,), torch.float32, "cuda:0")
    assert (t.made_on, t.recorded) == ("callers", [])


@pytest.mark.parametrize("likely", [0, 512])
def test_workspaces_are_the_calls_streams_alone(streams, monkeypatch, likely):
    """Both the workspace that a call is given first and the one that it then asks for."""
    seen = []
    monkeypatch.setattr(Tensor, "numel", lambda t: t.shape[0], raising=False)
    monkeypatch.setattr(Tensor, "element_size", lambda t: 1, raising=False)
    monkeypatch.setattr(Tensor, "data_ptr", lambda t: seen.append(t), raising=False)
    monkeypatch.setattr(binding, "_ptr", lambda t, *_: None if t is None else t.data_ptr())

    def call(address, size):
        if size._obj.value < 1024:
            size._obj.value = 1024
            return binding.CAPACITY
        return binding.OK

    binding._with_workspace(call, None, likely, "cuda:0", Stream("side"), "test")
    assert [(t.made_on, t.shape, t.recorded) for t in seen] == [("side", (n,), []) for n in (likely, 1024) if n]


def test_every_allocation_goes_through_it():
    with open(binding.__file__) as f:
        source = f.read()
    inside = source[source.index("def _empty("):source.index("def _check(")]
    assert len(re.findall(r"torch\.(empty|zeros|full|ones)\w*\(", source)) == len(re.findall(r"torch\.empty\(", inside)) == 2
