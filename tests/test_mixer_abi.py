"""Refusals of the selective scan, the causal convolution and the norm and rotation: before anything touches a GPU."""
import pytest
import torch

from mesa_layer_gb300 import binding, build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _scan(lib, **kw):
    a = dict(B=1, H=2, Hk=1, T=8, dk=16, dv=16, dtype=0, q=16, k=16, v=16, dt=16, A=16, bias=None, skip=None, starts=None,
             out=16, S0=None, Sf=None, ws=256, n=1 << 30)
    assert not set(kw) - set(a)
    return lib.mesa_ssm_forward_chunked(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(dtype=2), INVALID), (dict(H=3, Hk=2), INVALID), (dict(Hk=0), INVALID),
    (dict(dk=48), UNSUPPORTED), (dict(dv=8), UNSUPPORTED), (dict(B=40000, H=2), UNSUPPORTED), (dict(q=8), INVALID),
    (dict(out=24), INVALID), (dict(S0=8), INVALID), (dict(q=None), INVALID), (dict(dt=None), INVALID), (dict(A=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=128), WORKSPACE), (dict(B=0), OK),
    (dict(T=0), OK), (dict(T=0, S0=16, Sf=16), OK)])
def test_scan_refusals(lib, kw, want):
    assert _scan(lib, **kw) == want


def _scan_bwd(lib, **kw):
    a = dict(B=1, H=2, Hk=1, T=8, dk=16, dv=16, dtype=0, q=16, k=16, v=16, dt=16, A=16, bias=16, skip=16, starts=None, dout=16,
             S0=None, dSf=None, dq=16, dk_=16, dv_=16, ddt=16, dA=16, dbias=16, dskip=16, dS0=None, ws=256, n=1 << 30)
    assert not set(kw) - set(a)
    return lib.mesa_ssm_backward_chunked(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=512), INVALID), (dict(dk=48), UNSUPPORTED), (dict(bias=None), INVALID), (dict(skip=None), INVALID),
    (dict(dout=None), INVALID), (dict(dq=None), INVALID), (dict(ddt=None), INVALID), (dict(dv_=8), INVALID), (dict(dS0=8), INVALID),
    (dict(n=16), WORKSPACE), (dict(dtype=256, ws=None), WORKSPACE),
    (dict(T=0, dA=None, dbias=None, dskip=None), OK), (dict(B=0, dA=None, dbias=None, dskip=None), OK)])
def test_scan_backward_refusals(lib, kw, want):
    assert _scan_bwd(lib, **kw) == want


def test_scan_step_refusals(lib):
    def call(N=1, H=2, Hk=1, dk=16, dv=16, dtype=0, S=16, q=16, k=16, v=16, dt=16, A=16, out=16):
        return lib.mesa_ssm_step(N, H, Hk, dk, dv, dtype, S, q, k, v, dt, A, None, None, out, None)

    assert call(N=-1) == INVALID and call(dtype=3) == INVALID and call(H=3, Hk=2) == INVALID and call(dk=24) == UNSUPPORTED
    assert call(S=8) == INVALID and call(A=None) == INVALID and call(N=0) == OK and call(N=1 << 30, H=4) == UNSUPPORTED


def test_workspace_sizes(lib):
    f, b = lib.mesa_ssm_workspace_size, lib.mesa_ssm_backward_workspace_size
    assert f(1, 2, 1, 64, 16, 16, 0) > 0 and f(1, 2, 1, 64, 17, 16, 0) == 0 and f(1, 3, 2, 64, 16, 16, 0) == 0
    assert b(1, 2, 1, 64, 16, 16, 0) > f(1, 2, 1, 64, 16, 16, 0) and b(1, 2, 1, 64, 16, 16, 0) == b(1, 2, 1, 64, 16, 16, 256)
    assert b(1, 2, 1, 64, 16, 16, 0) > b(1, 2, 2, 64, 16, 16, 0)  # shared key heads: parts of their own
    assert lib.mesa_causal_conv_backward_workspace_size(1, 2, 64, 16, 4) >= 2 * 16 * 5 * 4
    assert lib.mesa_causal_conv_backward_workspace_size(1, 2, 64, 12, 4) == 0
    assert lib.mesa_qk_norm_rotary_backward_workspace_size(1, 2, 2, 64, 128) >= 2 * 128 * 4
    assert lib.mesa_qk_norm_rotary_backward_workspace_size(1, 2, 2, 64, 96) == 0


def _conv(lib, **kw):
    a = dict(B=1, H=2, T=8, d=16, W=4, dtype=0, silu=1, x=16, w=16, bias=None, starts=None, s0=None, sf=None, out=32)
    assert not set(kw) - set(a)
    return lib.mesa_causal_conv(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(dtype=7), INVALID), (dict(W=0), INVALID), (dict(d=0), INVALID), (dict(d=12), UNSUPPORTED),
    (dict(W=9), UNSUPPORTED), (dict(d=65544), UNSUPPORTED), (dict(B=40000), UNSUPPORTED), (dict(x=8), INVALID), (dict(s0=8), INVALID),
    (dict(out=16), INVALID), (dict(s0=64, sf=64), INVALID), (dict(w=None), INVALID), (dict(x=None), INVALID), (dict(T=0), OK),
    (dict(B=0), OK)])
def test_conv_refusals(lib, kw, want):
    assert _conv(lib, **kw) == want


def test_conv_step_and_backward_refusals(lib):
    def step(N=1, H=2, d=16, W=4, dtype=0, x=16, w=16, state=16, out=16):
        return lib.mesa_causal_conv_step(N, H, d, W, dtype, 1, x, w, None, state, out, None)

    assert step(N=-1) == INVALID and step(d=12) == UNSUPPORTED and step(W=9) == UNSUPPORTED and step(state=None) == INVALID
    assert step(N=0) == OK and step(x=8) == INVALID and step(H=-1) == INVALID and step(N=1 << 30, H=16) == UNSUPPORTED

    def back(B=1, H=2, T=8, d=16, W=4, x=16, dout=32, dx=48, dw=16, bias=16, db=16, ws=256, n=1 << 30):
        return lib.mesa_causal_conv_backward(B, H, T, d, W, 0, 1, x, 16, bias, None, dout, dx, dw, db, ws, n, None)

    assert back(dx=16) == INVALID and back(dx=32) == INVALID and back(bias=None) == INVALID and back(dout=8) == INVALID
    assert back(ws=None) == WORKSPACE and back(n=8) == WORKSPACE and back(T=0, dw=None, db=None) == OK


def test_rotary_refusals(lib):
    def call(B=1, H=2, Hk=1, T=8, d=16, R=16, dtype=0, norm=1, q=16, k=16, wq=None, f=16, off=0, scale=1.0, eps=1e-6, qo=16, ko=16):
        return lib.mesa_qk_norm_rotary(B, H, Hk, T, d, R, dtype, 0, norm, q, k, wq, None, f, None, off, scale, eps, qo, ko, None)

    assert call(B=-1) == INVALID and call(R=3) == INVALID and call(R=18) == INVALID and call(dtype=2) == INVALID
    assert call(eps=-1.0) == INVALID and call(scale=float("nan")) == INVALID and call(norm=0, wq=16) == INVALID
    assert call(d=24, R=0) == UNSUPPORTED and call(B=1 << 20, T=1 << 12) == UNSUPPORTED and call(off=0x7fffffff) == UNSUPPORTED
    assert call(f=None) == INVALID and call(k=None) == INVALID and call(qo=None) == INVALID and call(q=8) == INVALID
    assert call(T=0) == OK and call(H=0, Hk=0) == OK

    def back(T=8, dq_out=16, dq=16, wq=16, dwq=16, q=16, norm=1, ws=256, n=1 << 30):
        return lib.mesa_qk_norm_rotary_backward(1, 2, 0, T, 16, 16, 0, 0, norm, q, None, wq, None, 16, None, 0, 1.0, 1e-6, dq_out, None,
                                                dq, None, dwq, None, ws, n, None)

    assert back(wq=None) == INVALID and back(dq_out=None) == INVALID and back(q=None) == INVALID and back(ws=None) == WORKSPACE
    assert back(n=8) == WORKSPACE and back(T=0, dwq=None) == OK


def test_binding_refuses_host_tensors_and_shapes():
    q, v, dt, A = torch.zeros(1, 1, 4, 16), torch.zeros(1, 2, 4, 16), torch.zeros(1, 2, 4), torch.zeros(2)
    with pytest.raises(binding.MesaError, match="CUDA"):
        binding.mesa_ssm_forward_chunked(q, q, v, dt, A)
    with pytest.raises(binding.MesaError, match="CUDA"):
        binding.mesa_causal_conv(v, torch.zeros(2, 16, 4))
    with pytest.raises(binding.MesaError, match="CUDA"):
        binding.mesa_qk_norm_rotary(q, q)
    with pytest.raises(binding.MesaError, match=r"\[N, Hk, dk\]"):
        binding.mesa_ssm_step(v, q, q, v, dt, A)
    with pytest.raises(binding.MesaError, match=r"\[H, d, W\]"):
        binding.mesa_causal_conv_step(q, torch.zeros(2, 16, 4), None)
    with pytest.raises(binding.MesaError, match="float32 or bfloat16"):
        binding.mesa_qk_norm_rotary(q.half(), q)


def test_another_device_is_refused(monkeypatch):
    """Kernels go to the current device: tensors (or a stream) of another one are refused before the launch."""
    class Stream:
        cuda_stream, device_index = 7, 1

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 5 + i, raising=False)
    assert binding._launch_stream(None, torch.device("cuda", 0)) == 5
    with pytest.raises(binding.MesaError, match="current device"):
        binding._launch_stream(None, torch.device("cuda", 1))
    with pytest.raises(binding.MesaError, match="current device"):
        binding._launch_stream(Stream, torch.device("cuda", 0))
    Stream.device_index = 0
    assert binding._launch_stream(Stream, torch.device("cuda", 0)) == 7
