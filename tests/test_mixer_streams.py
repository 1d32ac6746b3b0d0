"""Scan, convolution and norm with rotation on a given stream: outputs and scratch come from that stream's memory, and
the launch goes to it (CPU: stand-ins for the tensors, the allocator and the library)."""
import contextlib

import pytest
import torch

from mesa_layer_gb300 import binding

F32, BF16 = torch.float32, torch.bfloat16


class Tensor:
    device, is_cuda = torch.device("cuda", 0), True

    def __init__(self, shape, dtype=BF16, stream=None):
        self.shape, self.dtype, self.stream, self.recorded = torch.Size(shape), dtype, stream, []

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.recorded.append(stream)


class Side:
    cuda_stream, device_index = 5, 0


class Library:
    """Every entry point succeeds and notes its last argument; sizes are 0."""

    def __init__(self):
        self.launches = []

    def __getattr__(self, name):
        def call(*args):
            if not name.endswith("_size"):
                self.launches.append((name, args[-1]))
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    current, made, library = ["current"], [], Library()

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(*shape, dtype=F32, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        made.append(Tensor(shape, dtype, current[-1]))
        return made[-1]

    monkeypatch.setattr(binding.torch.cuda, "stream", on)
    monkeypatch.setattr(binding.torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(binding.torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(binding.torch, "empty", empty)
    monkeypatch.setattr(binding.torch, "empty_like", lambda t: empty(t.shape, dtype=t.dtype))
    monkeypatch.setattr(binding, "load", lambda: library)
    return made, library.launches


def calls(stream):
    B, H, Hk, T, d, W = 2, 4, 2, 8, 16, 4
    qk, v, gate, head = Tensor((B, Hk, T, d)), Tensor((B, H, T, d)), Tensor((B, H, T), F32), Tensor((H,), F32)
    row, kv = Tensor((B, H, d)), Tensor((B, Hk, d))
    taps, bias, weight, inv = Tensor((H, d, W), F32), Tensor((H, d), F32), Tensor((d,), F32), Tensor((d // 2,), F32)
    on = dict(stream=stream)
    return {
        "mesa_ssm_forward_chunked": lambda f: f(qk, qk, v, gate, head, **on),
        "mesa_ssm_backward_chunked": lambda f: f(qk, qk, v, gate, head, v, dt_bias=head, skip=head, **on),
        "mesa_ssm_step": lambda f: f(Tensor((B, H, d, d), F32), kv, kv, row, Tensor((B, H), F32), head, **on),
        "mesa_causal_conv": lambda f: f(v, taps, bias, **on),
        "mesa_causal_conv_step": lambda f: f(row, taps, Tensor((B, H, W - 1, d), F32), bias, **on),
        "mesa_causal_conv_backward": lambda f: f(v, taps, v, bias, **on),
        "mesa_qk_norm_rotary": lambda f: f(v, qk, weight, weight, inv, **on),
        "mesa_qk_norm_rotary_backward": lambda f: f(v, qk, v, qk, weight, weight, inv, **on),
    }


@pytest.mark.parametrize("name", calls(None))
def test_memory_and_launch_are_the_streams(world, name):
    made, launches = world
    side = Side()
    calls(side)[name](getattr(binding, name))
    assert made and all(t.stream is side and t.recorded == ["current"] for t in made)
    assert launches == [(name, 5)]


@pytest.mark.parametrize("name", calls(None))
def test_a_stream_of_another_device_is_refused(world, name):
    class Other(Side):
        device_index = 1

    with pytest.raises(binding.MesaError, match="current device"):
        calls(Other())[name](getattr(binding, name))
    assert not world[1]
