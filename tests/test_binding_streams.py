"""Outputs and scratch of calls on a given stream come from that stream's memory (CPU: a recording
stand-in for the allocator)."""
import contextlib

import pytest
import torch

from mesa_layer_gb300 import binding


class Tensor:
    """Memory of a stream, or (stream None) a caller's fp32 CUDA tensor of the given shape."""
    device, is_cuda = "cuda:0", True

    def __init__(self, stream, shape=(1,), dtype=torch.float32):
        self.stream, self.shape, self.dtype, self.recorded = stream, shape, dtype, []

    def numel(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

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
    made = []

    def make(*args, **kwargs):
        made.append(Tensor(current[-1], dtype=kwargs.get("dtype", torch.float32)))
        return made[-1]

    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(binding.torch, name, make)
    return made


MAKE = {"_new": lambda s: binding._new((2, 3), None, "cuda:0", s), "_like": lambda s: binding._like(None, s),
        "_workspace": lambda s: binding._workspace(None, 1000, "cuda:0", s)}


@pytest.mark.parametrize("name", MAKE)
def test_memory_belongs_to_the_stream_that_uses_it(allocator, name):
    t = MAKE[name]("side")
    assert t.stream == "side"             # freed blocks of the current stream are not written early
    assert t.recorded == ["current"]      # and it may be used and freed there
    t = MAKE[name](None)
    assert t.stream == "current" and t.recorded == []


class Library:
    """Every entry point succeeds; sizes are 0."""

    def __getattr__(self, name):
        return lambda *args: 0


def _layer_calls(s):
    x, g, lam, taps = Tensor(None, (1, 2, 8, 16)), Tensor(None, (1, 2, 8)), Tensor(None, (2, 16)), Tensor(None, (2, 16, 4))
    row, gates, state = Tensor(None, (1, 2, 16)), Tensor(None, (1, 2)), Tensor(None, (1, 2, 16, 16))
    solve = (4, 0.0)
    return {
        "forward": lambda: binding.mesa_forward_chunked(x, x, x, g, lam, *solve, 64, stream=s),
        "forward_pre": lambda: binding.mesa_forward_chunked_pre(x, x, taps, taps, x, g, lam, *solve, 64, stream=s),
        "forward_save": lambda: binding.mesa_forward_chunked_save(x, x, x, g, lam, *solve, 64, stream=s),
        "forward_noalloc": lambda: binding.mesa_forward_chunked_noalloc(x, x, x, g, lam, *solve, 64, stream=s),
        "backward": lambda: binding.mesa_backward_chunked(x, x, x, g, lam, x, *solve, stream=s),
        "decode": lambda: binding.mesa_decode_step(state, state, row, row, row, gates, lam, *solve, stream=s),
        "decode_warm": lambda: binding.mesa_decode_step_warm(state, state, row, row, row, row, gates, lam, *solve, stream=s),
        "preprocess": lambda: binding.mesa_qk_preprocess(x, x, taps, taps, stream=s),
        "preprocess_step": lambda: binding.mesa_qk_preprocess_step(row, row, taps, taps, state, stream=s),
        "selftest": lambda: binding.mesa_tc_selftest(x, x, stream=s),
    }


@pytest.mark.parametrize("name", _layer_calls(None))
def test_the_layers_entry_points_on_a_given_stream(allocator, monkeypatch, name):
    class Side:
        cuda_stream = 5

    side = Side()
    monkeypatch.setattr(binding, "load", lambda: Library())
    _layer_calls(side)[name]()
    assert allocator and all(t.stream is side and t.recorded == ["current"] for t in allocator)
