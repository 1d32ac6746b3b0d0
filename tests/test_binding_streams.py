"""Outputs and scratch of calls on a given stream come from that stream's memory (CPU: a recording
stand-in for the allocator)."""
import contextlib

import pytest

from mesa_layer_gb300 import binding


class Tensor:
    device = "cuda:0"

    def __init__(self, stream):
        self.stream, self.recorded = stream, []

    def numel(self):
        return 1

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def allocator(monkeypatch):
    current = ["current"]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(binding.torch.cuda, "stream", on)
    monkeypatch.setattr(binding.torch.cuda, "current_stream", lambda device=None: current[-1])
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(binding.torch, name, lambda *a, **k: Tensor(current[-1]))


MAKE = {"_new": lambda s: binding._new((2, 3), None, "cuda:0", s), "_like": lambda s: binding._like(None, s),
        "_workspace": lambda s: binding._workspace(None, 1000, "cuda:0", s)}


@pytest.mark.parametrize("name", MAKE)
def test_memory_belongs_to_the_stream_that_uses_it(allocator, name):
    t = MAKE[name]("side")
    assert t.stream == "side"             # freed blocks of the current stream are not written early
    assert t.recorded == ["current"]      # and it may be used and freed there
    t = MAKE[name](None)
    assert t.stream == "current" and t.recorded == []
