"""The block norm on the GPU against the 64-bit restatement.  Tolerances on the 2-norm of each
output: fp32 -- a few products and a mean, each to 2^-24: 2e-6; sums over the rows 1e-5.  bf16 --
one rounding to 2^-9 (rms 1.7e-3): 3e-3; the weights' gradients stay fp32: 1e-5."""
import numpy as np
import pytest

import delta_reference as ref
from mesa_layer_gb300.synth import round_bf16

pytestmark = pytest.mark.gpu
TOL = {"f32": 2e-6, "bf16": 3e-3}
EPS = 1e-5
ALL = dict(x=1, gate=1, w_post=1, res_scale=1, w_pre=1)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mesa_layer_gb300 import binding, build
    build.build()
    binding.load()


def inputs(seed, dtype, N, D, parts, zero_row=False):
    r = np.random.default_rng(seed)
    rnd = round_bf16 if dtype == "bf16" else (lambda x: np.ascontiguousarray(x, dtype=np.float32))
    a = {n: rnd(r.standard_normal((N, D)) * (3.0 if n == "gate" else 1.0)) for n in ("x", "y", "gate", "dx_out", "dh")}
    if zero_row and N > 1:
        a["y"][1] = 0.0
        a["gate"][0] = -200.0  # a closed gate: e^200 overflows fp32
    a.update({n: (1.0 + 0.3 * r.standard_normal(D)).astype(np.float32) for n in ("w_post", "res_scale", "w_pre")})
    for n in ("x", "gate", "w_post", "res_scale", "w_pre"):
        if n not in parts:
            a[n] = None
    return a


def upload(a, dtype):
    import torch
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    return {n: None if x is None else torch.from_numpy(np.array(x)).cuda().to(
        torch.float32 if x.ndim == 1 else td) for n, x in a.items()}


def err(got, want):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape and np.isfinite(got).all()
    return np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)


CASES = [  # dtype, N, D, parts
    ("f32", 1, 1, ALL), ("f32", 3, 7, ALL), ("f32", 37, 64, dict(gate=1, w_post=1)), ("f32", 5, 130, dict(x=1)),
    ("f32", 9, 1000, ALL), ("f32", 4, 2048, dict(x=1, w_pre=1)), ("f32", 3, 8192, ALL), ("f32", 700, 100, ALL),
    ("bf16", 2, 16, ALL), ("bf16", 1300, 128, dict(gate=1, w_post=1)), ("bf16", 8, 2048, ALL), ("bf16", 5, 1001, ALL),
    ("bf16", 3, 1002, dict(x=1, w_post=1, res_scale=1, w_pre=1)), ("bf16", 3, 500, dict(w_post=1, w_pre=1)),
    ("bf16", 1400, 512, dict(x=1, gate=1, w_pre=1)), ("bf16", 2, 4097, ALL), ("bf16", 3, 8191, ALL),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}-{'+'.join(c[3])}")
def test_forward(case):
    from mesa_layer_gb300 import binding
    dtype, N, D, parts = case
    a = inputs(21, dtype, N, D, parts, zero_row=True)
    t = upload(a, dtype)
    X, h = binding.mesa_block_norm(t["x"], t["y"], t["gate"], t["w_post"], t["res_scale"], t["w_pre"], EPS)
    wX, wh = ref.norm_forward(a["x"], a["y"], a["gate"], a["w_post"], a["res_scale"], a["w_pre"], EPS)
    assert err(X, wX) <= TOL[dtype]
    assert (h is None) == (wh is None)
    if h is not None:
        assert err(h, wh) <= TOL[dtype]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}-{'+'.join(c[3])}")
def test_backward(case):
    from mesa_layer_gb300 import binding
    dtype, N, D, parts = case
    a = inputs(22, dtype, N, D, parts, zero_row=True)
    t = upload(a, dtype)
    names = ("dx", "dy", "dgate", "dw_post", "dres_scale", "dw_pre")
    got = dict(zip(names, binding.mesa_block_norm_backward(
        t["x"], t["y"], t["dx_out"], t["dh"], t["gate"], t["w_post"], t["res_scale"], t["w_pre"], EPS)))
    want = ref.norm_backward(a["x"], a["y"], a["gate"], a["w_post"], a["res_scale"], a["w_pre"], EPS, a["dx_out"],
                             a["dh"])
    for n in names:
        have = {"dx": "x", "dgate": "gate"}.get(n, n[1:])
        assert (got[n] is None) == (n != "dy" and have not in parts), n
        if got[n] is not None:
            assert err(got[n], want[n]) <= (1e-5 if n in ("dw_post", "dres_scale", "dw_pre") else 2 * TOL[dtype]), n


def test_gradient_against_differences_of_the_forward():
    import torch

    from mesa_layer_gb300 import binding
    a = inputs(23, "f32", 6, 96, ALL)
    t = upload(a, "f32")
    g = dict(zip(("x", "y", "gate", "w_post", "res_scale", "w_pre"), binding.mesa_block_norm_backward(
        t["x"], t["y"], t["dx_out"], t["dh"], t["gate"], t["w_post"], t["res_scale"], t["w_pre"], EPS)))
    gen = torch.Generator(device="cuda").manual_seed(3)
    for name in g:
        d = torch.randn(t[name].shape, generator=gen, device="cuda")
        step = 3e-3

        def loss(c):
            p = {**t, name: t[name] + c * d}
            X, h = binding.mesa_block_norm(p["x"], p["y"], p["gate"], p["w_post"], p["res_scale"], p["w_pre"], EPS)
            return ((X.double() * t["dx_out"].double()).sum() + (h.double() * t["dh"].double()).sum()).item()

        num = (loss(step) - loss(-step)) / (2 * step)
        ana = (g[name].double() * d.double()).sum().item()
        assert abs(num - ana) <= 2e-3 * (g[name].double().norm() * d.double().norm()).item(), (name, num, ana)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_missing_upstream_gradients_are_zero_and_in_place_forward(dtype):
    import torch

    from mesa_layer_gb300 import binding
    a = inputs(24, dtype, 33, 256, ALL)
    t = upload(a, dtype)
    w = dict(gate=t["gate"], w_post=t["w_post"], res_scale=t["res_scale"], w_pre=t["w_pre"], eps=EPS)
    zero = torch.zeros_like(t["y"])
    for dx_out, dh in ((None, t["dh"]), (t["dx_out"], None)):
        got = binding.mesa_block_norm_backward(t["x"], t["y"], dx_out, dh, **w)
        want = binding.mesa_block_norm_backward(t["x"], t["y"], zero if dx_out is None else dx_out,
                                                zero if dh is None else dh, **w)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    X, h = binding.mesa_block_norm(t["x"], t["y"], **w)
    x, y = t["x"].clone(), t["y"].clone()
    binding.mesa_block_norm(x, y, x_out=x, h_out=y, **w)
    assert torch.equal(x, X) and torch.equal(y, h)


def test_unaligned_rows_and_another_stream():
    """Views that start inside a vector (2 and 4 bytes off a 16-byte boundary) and a side stream."""
    import torch

    from mesa_layer_gb300 import binding
    base = torch.randn(3 * 640 + 8, device="cuda").to(torch.bfloat16)
    want = None
    side = torch.cuda.Stream()
    for off in (0, 1, 2):
        buf = torch.empty_like(base)
        y = buf[off:off + 3 * 640].view(3, 640)
        y.copy_(base[:3 * 640].view(3, 640))
        side.wait_stream(torch.cuda.current_stream())
        w = torch.ones(640, device="cuda")
        X, h = binding.mesa_block_norm(y, y, w_post=w, w_pre=w, stream=side if off else None)
        torch.cuda.current_stream().wait_stream(side)
        want = (X, h) if want is None else want
        # another split of the row over the lanes: the means may round differently
        assert (X.float() - want[0].float()).abs().max() <= 2 ** -7 * want[0].float().abs().max()
        assert (h.float() - want[1].float()).abs().max() <= 2 ** -7 * want[1].float().abs().max()


def test_writes_stay_inside_their_buffers():
    import torch

    from mesa_layer_gb300 import binding
    from test_gpu_canary import Guarded, workspace
    for dtype, N, D in (("bf16", 5, 1001), ("f32", 37, 60), ("bf16", 3, 2048)):
        a = inputs(25, dtype, N, D, ALL)
        t = upload(a, dtype)
        td = t["y"].dtype
        rows = [Guarded((N, D), td) for _ in range(5)]
        ws = workspace(binding.mesa_block_norm_backward_workspace_size(N, D))
        cols = [Guarded((D,), torch.float32) for _ in range(3)]
        w = dict(gate=t["gate"], w_post=t["w_post"], res_scale=t["res_scale"], w_pre=t["w_pre"], eps=EPS)
        binding.mesa_block_norm(t["x"], t["y"], x_out=rows[0].t, h_out=rows[1].t, **w)
        binding.mesa_block_norm_backward(t["x"], t["y"], t["dx_out"], t["dh"], dx=rows[2].t, dy=rows[3].t,
                                         dgate=rows[4].t, dw_post=cols[0].t, dres_scale=cols[1].t, dw_pre=cols[2].t,
                                         workspace=ws.t, **w)
        assert all(b.intact() for b in [*rows, *cols, ws])


def test_no_rows():
    import torch

    from mesa_layer_gb300 import binding
    y, w = torch.zeros(0, 48, device="cuda"), torch.ones(48, device="cuda")
    X, h = binding.mesa_block_norm(None, y, w_post=w, w_pre=w)
    assert X.shape == (0, 48) and h.shape == (0, 48)
    got = binding.mesa_block_norm_backward(None, y, y, y, w_post=w, w_pre=w)
    assert got[0] is None and not got[3].any() and not got[5].any()
