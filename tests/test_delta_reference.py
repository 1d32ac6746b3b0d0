"""CPU checks of the 64-bit restatements the GPU tests compare with: the gradients against
central differences, and special cases with known answers; the refusals of the gated delta rule's
and the block norm's entry points (every one before the GPU is touched)."""
import ctypes

import numpy as np
import pytest

import delta_reference as ref
from mesa_layer_gb300 import binding, build

EPS = 1e-6  # difference step: truncation ~ step^2, rounding ~ 2^-53 / step = 1e-10 of the value


def test_rule_gradients_against_differences():
    s = ref.rule_inputs(3, "f32", 1, 4, 2, 9, 16, 16, gates="packed", S0=True)
    s["gamma"][0, 1, 4] = 0.0
    g = ref.rule_backward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], 0.7, s["dout"], s["S0"], s["dS_final"])
    r = np.random.default_rng(1)

    def loss(x):
        o, S = ref.rule_forward(x["q"], x["k"], x["v"], x["gamma"], x["beta"], 0.7, x["S0"])
        return (o * s["dout"]).sum() + (S * s["dS_final"]).sum()

    for name in ("q", "k", "v", "gamma", "beta", "S0"):
        d = r.standard_normal(s[name].shape)
        up, dn = dict(s), dict(s)
        up[name] = s[name].astype(np.float64) + EPS * d
        dn[name] = s[name].astype(np.float64) - EPS * d
        num = (loss(up) - loss(dn)) / (2 * EPS)
        ana = (g["d" + name] * d).sum()
        assert abs(num - ana) <= 1e-6 * (1 + abs(ana)), name


def test_rule_special_cases():
    s = ref.rule_inputs(4, "f32", 1, 2, 2, 5, 16, 16, gates="shut")
    o, _ = ref.rule_forward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], 1.0)
    qk = (s["q"].astype(np.float64) * s["k"]).sum(-1)  # every gate closed: the token's own write
    assert np.allclose(o, (s["beta"] * qk)[..., None] * s["v"], atol=1e-12)
    s = ref.rule_inputs(5, "f32", 1, 1, 1, 3, 16, 16, gates="one")
    s["k"][:] = s["k"][:, :, :1]  # one unit key, beta 1: the last value replaces the others
    o, S = ref.rule_forward(s["k"], s["k"], s["v"], s["gamma"], s["beta"], 1.0)
    assert np.allclose(o, s["v"], atol=1e-6)


def test_norm_gradients_against_differences():
    r = np.random.default_rng(7)
    N, D = 3, 10
    a = {n: r.standard_normal((N, D)) for n in ("x", "y", "gate", "dx_out", "dh")}
    w = {n: r.standard_normal(D) for n in ("w_post", "res_scale", "w_pre")}
    g = ref.norm_backward(a["x"], a["y"], a["gate"], w["w_post"], w["res_scale"], w["w_pre"], 1e-6, a["dx_out"], a["dh"])

    def loss(p):
        X, h = ref.norm_forward(p["x"], p["y"], p["gate"], p["w_post"], p["res_scale"], p["w_pre"], 1e-6)
        return (X * a["dx_out"]).sum() + (h * a["dh"]).sum()

    base = {**a, **w}
    for name in ("x", "y", "gate", "w_post", "res_scale", "w_pre"):
        d = r.standard_normal(base[name].shape)
        num = (loss({**base, name: base[name] + EPS * d}) - loss({**base, name: base[name] - EPS * d})) / (2 * EPS)
        ana = (g["d" + name] * d).sum()
        assert abs(num - ana) <= 1e-6 * (1 + abs(ana)), name


# ---- refusals ---------------------------------------------------------------------------------
P = ctypes.c_void_p(1 << 20)   # a 16-byte aligned address that is never read
ODD = ctypes.c_void_p((1 << 20) + 4)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def fwd(lib, B=1, H=2, Hk=2, T=8, dk=64, dv=64, dtype=0, q=P, k=P, v=P, gamma=P, beta=P, scale=1.0, out=P, S0=None,
        SF=None, ws=P, nbytes=BIG):
    return lib.mesa_delta_forward_chunked(B, H, Hk, T, dk, dv, dtype, q, k, v, gamma, beta, scale, out, S0, SF, ws,
                                          nbytes, None)


def bwd(lib, B=1, H=2, Hk=2, T=8, dk=64, dv=64, dtype=0, q=P, dout=P, dq=P, dbeta=P, dS0=None, ws=P, nbytes=BIG):
    return lib.mesa_delta_backward_chunked(B, H, Hk, T, dk, dv, dtype, q, P, P, P, P, 1.0, dout, None, None, dq, P, P,
                                           P, dbeta, dS0, ws, nbytes, None)


def step(lib, N=1, H=2, Hk=2, dk=64, dv=64, dtype=0, S=P, q=P, out=P, scale=1.0):
    return lib.mesa_delta_step(N, H, Hk, dk, dv, dtype, S, q, P, P, P, P, scale, out, None)


def test_rule_refusals(lib):
    INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
    for call in (fwd, bwd, step):
        assert call(lib, H=3, Hk=2) == INVALID
        assert call(lib, H=2, Hk=0) == INVALID
        assert call(lib, H=-1) == INVALID
        assert call(lib, dtype=2) == INVALID
        assert call(lib, dk=48) == UNSUPPORTED
        assert call(lib, dv=256) == UNSUPPORTED
        assert call(lib, q=None) == INVALID
        assert call(lib, q=ODD) == INVALID
    for call in (fwd, bwd):
        assert call(lib, T=-1) == INVALID
        assert call(lib, B=65536, H=1, Hk=1) == UNSUPPORTED
        assert call(lib, ws=None) == WORKSPACE
        assert call(lib, nbytes=16) == WORKSPACE
        assert call(lib, ws=ctypes.c_void_p((1 << 20) + 16)) == WORKSPACE
        assert call(lib, B=0) == 0 and call(lib, T=0) == 0
    for bad in (float("nan"), float("inf")):
        assert fwd(lib, scale=bad) == INVALID and step(lib, scale=bad) == INVALID
    for name in ("k", "v", "gamma", "beta", "out"):
        assert fwd(lib, **{name: None}) == INVALID
    for name in ("v", "out", "S0", "SF"):
        assert fwd(lib, **{name: ODD}) == INVALID
    for name in ("dout", "dq", "dbeta"):
        assert bwd(lib, **{name: None}) == INVALID
    for name in ("dout", "dq", "dS0"):
        assert bwd(lib, **{name: ODD}) == INVALID
    assert step(lib, S=None) == INVALID and step(lib, S=ODD) == INVALID and step(lib, out=None) == INVALID
    assert step(lib, N=0) == 0
    assert lib.mesa_delta_workspace_size(1, 3, 2, 8, 64, 64, 0) == 0
    assert lib.mesa_delta_backward_workspace_size(1, 2, 2, 8, 64, 24, 0) == 0


def test_norm_refusals(lib):
    INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3

    def f(N=2, D=64, dtype=0, x=P, y=P, gate=P, wp=P, rs=P, wn=P, eps=1e-6, xo=P, ho=P):
        return lib.mesa_block_norm(N, D, dtype, x, y, gate, wp, rs, wn, eps, xo, ho, None)

    assert f(N=-1) == INVALID and f(D=0) == INVALID and f(dtype=7) == INVALID
    assert f(D=8193) == UNSUPPORTED
    assert f(y=None) == INVALID and f(ho=None) == INVALID and f(xo=None, wn=None) == INVALID
    assert f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID
    assert f(N=0) == 0

    def b(N=2, D=64, dtype=0, y=P, gate=P, wp=P, rs=P, wn=P, dy=P, dgate=P, dwp=P, drs=P, dwn=P, ws=P, nbytes=BIG):
        return lib.mesa_block_norm_backward(N, D, dtype, P, y, gate, wp, rs, wn, 1e-6, P, P, P, dy, dgate, dwp, drs,
                                            dwn, ws, nbytes, None)

    assert b(y=None) == INVALID and b(dy=None) == INVALID and b(D=9000) == UNSUPPORTED
    assert b(gate=None) == INVALID and b(wp=None) == INVALID and b(rs=None) == INVALID and b(wn=None) == INVALID
    assert b(ws=None) == WORKSPACE and b(nbytes=64) == WORKSPACE
    assert lib.mesa_block_norm_backward_workspace_size(5, 8193) == 0


def test_the_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros(1, 2, 4, 16)
    g = torch.zeros(1, 2, 4)
    with pytest.raises(binding.MesaError):
        binding.mesa_delta_forward_chunked(x, x, x, g, g)
    with pytest.raises(binding.MesaError):
        binding.mesa_block_norm(None, x)
