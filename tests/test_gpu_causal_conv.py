"""The causal convolution on the GPU against its 64-bit form.

Tolerances on the 2-norm.  fp32: at most eight products and SiLU by the hardware's exponential and division (2^-21): 2^-18.
bf16: the output's rounding, 2^-8.  Sums over batch and time: fp32 sums of up to a few thousand terms, in runs of 32 and
trees of them: 2^-16 of the terms' 2-norm times sqrt of their number at worst, measured on that."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import off

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 2.0 ** -18, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mesa_layer_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def make(dtype, B, H, T, d, W, seed=0, packed=False, bias=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)

    s = dict(x=normal(B, H, T, d).to(dtype), w=W ** -0.5 * normal(H, d, W), bias=0.3 * normal(H, d) if bias else None,
             starts=torch.rand(B, T, generator=g) < 0.15 if packed else None, state0=normal(B, H, W - 1, d),
             dout=normal(B, H, T, d).to(dtype))
    return {n: None if t is None else t.cuda() for n, t in s.items()}


def double(t):
    return None if t is None else t.double()


CASES = [(1, 1, 1, 8, 1), (1, 1, 1, 8, 4), (2, 3, 2, 16, 8), (1, 2, 33, 64, 4), (2, 1, 100, 128, 3), (1, 5, 65, 24, 2), (2, 2, 257, 128, 4),
         (1, 1, 70, 520, 4), (3, 2, 31, 32, 5), (1, 1, 40, 1024, 7), (1, 2, 64, 8, 6)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("silu,packed,state", [(True, False, False), (False, True, False), (True, True, True)])
@pytest.mark.parametrize("B,H,T,d,W", CASES)
def test_forward(lib, dtype, silu, packed, state, B, H, T, d, W):
    s = make(dtype, B, H, T, d, W, seed=T, packed=packed, bias=silu)
    end = torch.full((B, H, W - 1, d), torch.nan, device="cuda")
    out = lib.mesa_causal_conv(s["x"], s["w"], bias=s["bias"], silu=silu, starts=s["starts"], state0=s["state0"] if state else None,
                               state_final=end)
    want, want_end = ref.conv(s["x"].double(), s["w"].double(), double(s["bias"]), silu, s["starts"],
                              s["state0"].double() if state else None)
    assert off(out, want) <= TOL[dtype]
    if W > 1:
        assert torch.equal(end.double(), want_end)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("silu,packed", [(True, False), (False, False), (True, True)])
@pytest.mark.parametrize("B,H,T,d,W", CASES)
def test_backward(lib, dtype, silu, packed, B, H, T, d, W):
    s = make(dtype, B, H, T, d, W, seed=T + 1, packed=packed)
    x, w, b = (s[n].double().requires_grad_() for n in ("x", "w", "bias"))
    out, _ = ref.conv(x, w, b, silu, s["starts"])
    (out * s["dout"].double()).sum().backward()
    dx, dw, db = lib.mesa_causal_conv_backward(s["x"], s["w"], s["dout"], bias=s["bias"], silu=silu, starts=s["starts"])
    assert off(dx, x.grad) <= TOL[dtype]
    size = float((s["dout"].double().square().sum() * (1 + s["x"].double().square().mean())).sqrt())
    for got, want in ((dw, w.grad), (db, b.grad)):
        assert float((got.double() - want).norm()) <= 2.0 ** -16 * max(size, float(want.norm()))
    again = lib.mesa_causal_conv_backward(s["x"], s["w"], s["dout"], bias=s["bias"], silu=silu, starts=s["starts"])
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)
    if silu:  # without a bias, a starts array that marks nothing
        r = lib.mesa_causal_conv_backward(s["x"], s["w"], s["dout"], silu=False, starts=torch.zeros_like(s["x"][:, 0, :, 0], dtype=torch.uint8))
        p = lib.mesa_causal_conv_backward(s["x"], s["w"], s["dout"], silu=False)
        assert r[2] is None and all(torch.equal(i, j) for i, j in zip(r[:2], p[:2]))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,H,d,W", [(1, 1, 8, 1), (1, 4, 128, 4), (7, 3, 64, 2), (2, 1, 1000, 8)])
def test_step_goes_on_from_a_prompt(lib, dtype, N, H, d, W):
    T, more = 5, 3
    s = make(dtype, N, H, T + more, d, W, seed=d)
    state = torch.empty(N, H, W - 1, d, device="cuda")
    lib.mesa_causal_conv(s["x"][:, :, :T].contiguous(), s["w"], bias=s["bias"], state_final=state)
    outs = [lib.mesa_causal_conv_step(s["x"][:, :, T + i].contiguous(), s["w"], state if W > 1 else None, bias=s["bias"])
            for i in range(more)]
    want, end = ref.conv(s["x"].double(), s["w"].double(), s["bias"].double())
    assert off(torch.stack(outs, 2), want[:, :, T:]) <= TOL[dtype]
    if W > 1:
        assert torch.equal(state.double(), end)
    x = s["x"][:, :, 0].contiguous()
    a, b = state.clone(), state.clone()
    o = lib.mesa_causal_conv_step(x, s["w"], a if W > 1 else None, bias=s["bias"])
    lib.mesa_causal_conv_step(x, s["w"], b if W > 1 else None, bias=s["bias"], out=x)  # in place
    assert torch.equal(o, x) and torch.equal(a, b)


def test_nothing_beyond_and_empty(lib):
    s = make(BF16, 1, 2, 37, 24, 4)
    n = 2 * 37 * 24
    room = torch.full((n + 512,), 3.0, dtype=BF16, device="cuda")
    out = lib.mesa_causal_conv(s["x"], s["w"], bias=s["bias"], out=room[:n].view(1, 2, 37, 24))
    assert torch.equal(out, lib.mesa_causal_conv(s["x"], s["w"], bias=s["bias"])) and bool((room[n:] == 3).all())
    e = s["x"][:, :, :0].contiguous()
    end = torch.empty(1, 2, 3, 24, device="cuda")
    assert lib.mesa_causal_conv(e, s["w"], state0=s["state0"], state_final=end).shape == e.shape and torch.equal(end, s["state0"])
    dx, dw, db = lib.mesa_causal_conv_backward(e, s["w"], e, bias=s["bias"])
    assert dx.shape == e.shape and not dw.any() and not db.any()


def test_a_nan_before_a_start_stays_there(lib):
    s = make(F32, 1, 1, 20, 8, 4)
    s["starts"] = torch.zeros(1, 20, dtype=torch.bool, device="cuda")
    s["starts"][0, 10] = True
    clean = lib.mesa_causal_conv(s["x"], s["w"], starts=s["starts"])
    s["x"][0, 0, 9] = torch.nan
    out = lib.mesa_causal_conv(s["x"], s["w"], starts=s["starts"])
    assert torch.equal(out[:, :, 10:], clean[:, :, 10:]) and torch.equal(out[:, :, :9], clean[:, :, :9])
    dx, _, _ = lib.mesa_causal_conv_backward(s["x"], s["w"], s["dout"], starts=s["starts"])
    assert torch.isfinite(dx[:, :, 10:]).all()


def test_captured(lib):
    s, t = make(BF16, 2, 2, 90, 64, 4, seed=1), make(BF16, 2, 2, 90, 64, 4, seed=2)
    want = lib.mesa_causal_conv(t["x"], t["w"], bias=t["bias"])
    wg = lib.mesa_causal_conv_backward(t["x"], t["w"], t["dout"], bias=t["bias"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.mesa_causal_conv(s["x"], s["w"], bias=s["bias"])
        g = lib.mesa_causal_conv_backward(s["x"], s["w"], s["dout"], bias=s["bias"])
    for n in ("x", "w", "bias", "dout"):
        s[n].copy_(t[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(i, j) for i, j in zip(g, wg))
