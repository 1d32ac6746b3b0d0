"""The selective state space scan on the GPU against its 64-bit token recurrence.

Tolerances, relative on the 2-norm of each output.  fp32: every value is a sum of a few hundred products, each rounded to
2^-24; their errors add up to at most 256 2^-24 = 2^-16 of the terms.  bf16: the output's rounding is at most 2^-8 of a
value, and two operands of each product (the pairs' weights, the state; in a gradient's inner products one more) are
rounded as much: 3 2^-8, gradients 4 2^-8.  fp32 states of bf16 inputs: weights as two bf16 values, 2^-16 of each term,
beside the fp32 sums: 2^-15.  Sums of gradients over a head's tokens are measured on the norm over the heads of the
terms' own sizes (sqrt of the sum of squares of the per-token values), as the sum may cancel: the same bounds."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import off

pytestmark = pytest.mark.gpu
TOL = {torch.float32: 2.0 ** -16, torch.bfloat16: 3 * 2.0 ** -8}
GRAD_TOL = {torch.float32: 2.0 ** -15, torch.bfloat16: 4 * 2.0 ** -8}
STATE_TOL = {torch.float32: 2.0 ** -16, torch.bfloat16: 2.0 ** -15}
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mesa_layer_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def make(dtype, B, H, Hk, T, dk, dv, seed=0, packed=False, states=False, steps=(1e-3, 0.3), bias=True, skip=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)

    lo, hi = (torch.tensor(x).log() for x in steps)
    step = torch.exp(lo + (hi - lo) * torch.rand(H, generator=g))
    b = step + torch.log(-torch.expm1(-step))
    s = dict(q=dk ** -0.5 * normal(B, Hk, T, dk), k=normal(B, Hk, T, dk), v=normal(B, H, T, dv), dt=0.7 * normal(B, H, T),
             A=-1.0 - 15.0 * torch.rand(H, generator=g), dt_bias=b if bias else None,
             skip=1 + 0.1 * normal(H) if skip else None, starts=None, S0=None, dout=normal(B, H, T, dv), dS_final=None)
    if not bias:
        s["dt"] = s["dt"] + b[:, None]
    if packed:
        s["starts"] = torch.rand(B, T, generator=g) < 0.03
        s["dt"][:, :, T - T // 8:] = -torch.inf
    if states:
        s["S0"], s["dS_final"] = normal(B, H, dv, dk), normal(B, H, dv, dk)
    for n in ("q", "k", "v", "dout"):
        s[n] = s[n].to(dtype)
    return {n: None if x is None else x.cuda() for n, x in s.items()}


def exact(s, grads=False):
    x = {n: None if s[n] is None else s[n].double() for n in ("q", "k", "v", "dt", "A", "dt_bias", "skip", "S0")}
    if grads:
        x = {n: None if t is None else t.requires_grad_() for n, t in x.items()}
    out, S = ref.scan(x["q"], x["k"], x["v"], x["dt"], x["A"], x["dt_bias"], x["skip"], s["starts"], x["S0"])
    if not grads:
        return out, S
    L = (out * s["dout"].double()).sum()
    if s["dS_final"] is not None:
        L = L + (S * s["dS_final"].double()).sum()
    L.backward()
    return {n: t.grad for n, t in x.items() if t is not None}


def forward(lib, s, **kw):
    S = torch.full(s["v"].shape[:2] + (s["v"].shape[-1], s["q"].shape[-1]), torch.nan, device="cuda")
    out = lib.mesa_ssm_forward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], dt_bias=s["dt_bias"], skip=s["skip"],
                                       starts=s["starts"], S0=s["S0"], S_final=S, **kw)
    return out, S


SIZES = [  # dtype, B, H, Hk, T, dk, dv, packed, states
    (F32, 1, 1, 1, 1, 16, 16, False, True), (F32, 2, 3, 1, 33, 16, 64, True, True), (F32, 1, 4, 2, 70, 32, 16, False, False),
    (F32, 2, 4, 1, 257, 64, 64, True, True), (F32, 1, 2, 2, 100, 128, 64, False, True), (F32, 1, 2, 1, 65, 128, 128, True, False),
    (F32, 1, 3, 3, 600, 64, 32, False, True),
    (BF16, 2, 2, 1, 47, 64, 64, True, True), (BF16, 1, 2, 2, 31, 32, 128, False, False), (BF16, 1, 1, 1, 1, 128, 128, False, True),
    (BF16, 1, 2, 2, 2, 128, 64, False, False), (BF16, 2, 4, 2, 127, 128, 128, True, True), (BF16, 1, 2, 2, 128, 128, 128, False, True),
    (BF16, 1, 3, 1, 129, 128, 64, False, True), (BF16, 2, 2, 2, 333, 128, 128, True, True), (BF16, 1, 2, 1, 700, 128, 64, True, False),
    (BF16, 1, 2, 2, 640, 128, 128, False, True), (BF16, 1, 2, 2, 300, 64, 128, False, True), (BF16, 1, 4, 2, 300, 64, 64, True, True), (BF16, 1, 2, 2, 129, 64, 64, False, True),
    (BF16, 2, 3, 3, 1500, 64, 64, True, True), (BF16, 1, 2, 1, 200, 128, 32, False, True), (BF16, 1, 1, 1, 3000, 128, 128, True, True),
]


def name(c):
    return f"{'f32' if c[0] is F32 else 'bf16'}-{c[1]}x{c[2]}({c[3]})x{c[4]}-{c[5]}x{c[6]}{'-packed' * c[7]}{'-states' * c[8]}"


@pytest.mark.parametrize("c", SIZES, ids=name)
def test_forward(lib, c):
    dtype, B, H, Hk, T, dk, dv, packed, states = c
    s = make(dtype, B, H, Hk, T, dk, dv, seed=T, packed=packed, states=states)
    out, S = forward(lib, s)
    want, want_S = exact(s)
    assert out.dtype == dtype and off(out, want) <= TOL[dtype]
    assert off(S, want_S) <= STATE_TOL[dtype]
    again, S2 = forward(lib, s)
    assert torch.equal(out, again) and torch.equal(S, S2)


@pytest.mark.parametrize("c", SIZES, ids=name)
def test_backward(lib, c):
    dtype, B, H, Hk, T, dk, dv, packed, states = c
    s = make(dtype, B, H, Hk, T, dk, dv, seed=T + 1, packed=packed, states=states)
    want = exact(s, grads=True)
    dS0 = torch.full((B, H, dv, dk), torch.nan, device="cuda") if states else None
    args = dict(dt_bias=s["dt_bias"], skip=s["skip"], starts=s["starts"], S0=s["S0"], dS_final=s["dS_final"], gates_dtype=F32)
    got = dict(zip(("q", "k", "v", "dt", "A", "dt_bias", "skip"), lib.mesa_ssm_backward_chunked(
        s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], dS0=dS0, **args)))
    for n in ("q", "k", "v", "dt"):
        assert off(got[n], want[n]) <= GRAD_TOL[dtype], n
    # a head's sums, on the size of its terms
    step = torch.nn.functional.softplus((s["dt"] + s["dt_bias"][:, None]).double())
    terms = {"dt_bias": want["dt"], "skip": s["dout"].double() * s["v"].double(), "A": want["dt"].abs() + step}
    for n, t in terms.items():
        size = t.square().sum() ** 0.5
        assert float((got[n].double() - want[n]).norm()) <= GRAD_TOL[dtype] * max(float(size), float(want[n].norm())), n
    if states:
        assert off(dS0, want["S0"]) <= STATE_TOL[dtype]
    rounded = lib.mesa_ssm_backward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], **{**args, "gates_dtype": dtype})
    for n, x in zip(("q", "k", "v", "dt", "A", "dt_bias", "skip"), rounded):
        assert x.dtype == dtype and torch.equal(x, got[n].to(dtype)), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,H,Hk,dk,dv", [(1, 1, 1, 16, 16), (3, 4, 2, 128, 128), (5, 2, 2, 64, 32), (2, 3, 1, 32, 128), (2, 2, 2, 128, 64)])
def test_step_goes_on_from_a_prompt(lib, dtype, N, H, Hk, dk, dv):
    T, more = 40, 3
    s = make(dtype, N, H, Hk, T + more, dk, dv, seed=dk + dv)
    want, want_S = exact(s)
    head = {n: x[:, :, :T].contiguous() if n in ("q", "k", "v", "dt") else x for n, x in s.items()}
    _, S = forward(lib, head)
    outs = [lib.mesa_ssm_step(S, *(s[n][:, :, T + i].contiguous() for n in ("q", "k", "v", "dt")), s["A"], dt_bias=s["dt_bias"],
                              skip=s["skip"]) for i in range(more)]
    assert off(torch.stack(outs, 2), want[:, :, T:]) <= TOL[dtype]
    assert off(S, want_S) <= STATE_TOL[dtype]


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF16, 128)])
def test_continued_in_pieces(lib, dtype, d):
    s = make(dtype, 2, 2, 2, 450, d, d, seed=5)
    out, S = forward(lib, s)
    state, outs = None, []
    for a, b in ((0, 130), (130, 131), (131, 450)):
        piece = {n: x[:, :, a:b].contiguous() if n in ("q", "k", "v", "dt") else x for n, x in s.items()}
        piece["S0"] = state
        o, state = forward(lib, piece)
        outs.append(o)
    assert off(torch.cat(outs, 2), out) <= TOL[dtype] and off(state, S) <= STATE_TOL[dtype]


@pytest.mark.parametrize("dtype,d", [(F32, 32), (BF16, 128)])
@pytest.mark.parametrize("steps", [(1e-6, 1e-5), (5.0, 50.0), (1e-4, 20.0)])
def test_hardly_and_very_forgetful_heads(lib, dtype, d, steps):
    """Steps of 1e-5 (nothing is forgotten over the sequence) and of 50 (log-decays of -800 a token)."""
    s = make(dtype, 1, 4, 4, 300, d, d, seed=9, steps=steps, states=True)
    out, S = forward(lib, s)
    want, want_S = exact(s)
    assert off(out, want) <= TOL[dtype] and off(S, want_S) <= STATE_TOL[dtype]
    got = lib.mesa_ssm_backward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], dt_bias=s["dt_bias"], skip=s["skip"],
                                        S0=s["S0"], dS_final=s["dS_final"], gates_dtype=F32)
    g = exact(s, grads=True)
    for n, x in zip(("q", "k", "v", "dt"), got):
        assert off(x, g[n]) <= GRAD_TOL[dtype], n


@pytest.mark.parametrize("dtype,d", [(F32, 32), (BF16, 128)])
def test_a_sudden_reset_keeps_the_neighbours_decays(lib, dtype, d):
    """One step of 1e6 among small ones: the differences of log-decays after it stay exact."""
    s = make(dtype, 1, 2, 2, 200, d, d, seed=11, steps=(1e-2, 1e-1))
    s["dt"][:, :, 70] = 1e6
    s["v"][:, :, 70] = 0
    out, S = forward(lib, s)
    want, want_S = exact(s)
    assert off(out, want) <= TOL[dtype] and off(S, want_S) <= STATE_TOL[dtype]


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF16, 128)])
def test_empty_sequences(lib, dtype, d):
    s = make(dtype, 2, 2, 1, 0, d, d, states=True)
    out, S = forward(lib, s)
    assert out.shape == (2, 2, 0, d) and torch.equal(S, s["S0"])
    dS0 = torch.empty_like(S)
    r = lib.mesa_ssm_backward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], dt_bias=s["dt_bias"], skip=s["skip"],
                                      dS_final=s["dS_final"], dS0=dS0)
    assert torch.equal(dS0, s["dS_final"]) and all(not x.float().abs().sum() for x in r[4:])


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF16, 64), (BF16, 128)])
def test_status_and_units_of_their_own(lib, dtype, d):
    """A NaN is reported and reaches its own unit's later tokens alone."""
    s = make(dtype, 2, 2, 2, 300, d, d, seed=3)
    ws = torch.empty(lib.mesa_ssm_workspace_size(2, 2, 2, 300, d, d, dtype), dtype=torch.uint8, device="cuda")
    out, _ = forward(lib, s, workspace=ws)
    assert lib.mesa_forward_status_code(ws)[0] == lib.MESA_OK
    s["v"][1, 0, 200, 3] = torch.nan
    out2, _ = forward(lib, s, workspace=ws)
    assert lib.mesa_forward_status_code(ws)[0] == lib.MESA_ERR_NONFINITE
    assert torch.equal(out[0], out2[0]) and torch.equal(out[1, 1], out2[1, 1]) and torch.equal(out[1, 0, :128], out2[1, 0, :128])
    assert out2[1, 0, 200:, 3].isnan().all()


@pytest.mark.parametrize("dtype,d", [(F32, 32), (BF16, 64), (BF16, 128)])
def test_gradients_of_units_of_their_own(lib, dtype, d):
    """A NaN in one unit's value is reported and reaches no other unit's gradients."""
    B, H, T = 2, 90, 200  # (more chunks than SMs: a CTA takes several units)
    s = make(dtype, B, H, H, T, d, d, seed=6)
    args = dict(dt_bias=s["dt_bias"], skip=s["skip"], gates_dtype=F32)
    ws = torch.empty(lib.mesa_ssm_backward_workspace_size(B, H, H, T, d, d, dtype), dtype=torch.uint8, device="cuda")
    clean = lib.mesa_ssm_backward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], workspace=ws, **args)
    assert lib.mesa_forward_status_code(ws)[0] == lib.MESA_OK
    s["v"][0, 3, 17, 5] = torch.nan
    r = lib.mesa_ssm_backward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], workspace=ws, **args)
    assert lib.mesa_forward_status_code(ws)[0] == lib.MESA_ERR_NONFINITE
    others = torch.ones(B, H, dtype=torch.bool, device="cuda")
    others[0, 3] = False
    assert all(torch.equal(x[others], y[others]) for x, y in zip(clean[:4], r[:4]))


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF16, 64), (BF16, 128)])
def test_states_in_place_and_nothing_beyond(lib, dtype, d):
    """S_final may be S0's memory; what lies behind each output stays."""
    B, H, T = 1, 3, 261
    s = make(dtype, B, H, H, T, d, d, seed=21, states=True)
    out, S = forward(lib, s)
    n, pad = B * H * T * d, 4096
    room = torch.full((n + pad,), 7.0, dtype=dtype, device="cuda")
    state = s["S0"].clone()
    o = lib.mesa_ssm_forward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], dt_bias=s["dt_bias"], skip=s["skip"],
                                     S0=state, S_final=state, out=room[:n].view(B, H, T, d))
    assert torch.equal(o, out) and torch.equal(state, S) and bool((room[n:] == 7.0).all())


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF16, 128)])
def test_captured_and_on_another_stream(lib, dtype, d):
    s, t = make(dtype, 1, 2, 2, 400, d, d, seed=31), make(dtype, 1, 2, 2, 400, d, d, seed=32)
    want, want_S = forward(lib, t)
    ws = torch.empty(lib.mesa_ssm_workspace_size(1, 2, 2, 400, d, d, dtype), dtype=torch.uint8, device="cuda")
    out, S = torch.empty_like(want), torch.empty_like(want_S)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call(**kw):
        return lib.mesa_ssm_forward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], dt_bias=s["dt_bias"], skip=s["skip"], **kw)

    with torch.cuda.stream(side):
        call(out=out, S_final=S, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out, S_final=S, workspace=ws)
    for n in ("q", "k", "v", "dt", "A", "dt_bias", "skip"):
        s[n].copy_(t[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(S, want_S)
    o = call(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, want)


@pytest.mark.parametrize("dk,d", [(128, 64), (128, 128), (64, 64)])
@pytest.mark.parametrize("T", [200, 6000])
def test_waits_that_give_up_are_reported(lib, dk, d, T):
    """On the tensor cores (whole sequences, and in segments): the status says so, the next call is clean."""
    s = make(BF16, 1, 2, 1, T, dk, d, seed=41, states=True)
    out, S = forward(lib, s)
    args = dict(dt_bias=s["dt_bias"], skip=s["skip"], S0=s["S0"], dS_final=s["dS_final"], gates_dtype=F32)
    scan = (s["q"], s["k"], s["v"], s["dt"], s["A"])
    grads = lib.mesa_ssm_backward_chunked(*scan, s["dout"], **args)
    ws = torch.empty(lib.mesa_ssm_workspace_size(1, 2, 1, T, dk, d, BF16), dtype=torch.uint8, device="cuda")
    wb = torch.empty(lib.mesa_ssm_backward_workspace_size(1, 2, 1, T, dk, d, BF16), dtype=torch.uint8, device="cuda")
    try:
        lib.mesa_debug_set_wait_limit(0)
        forward(lib, s, workspace=ws)
        lib.mesa_ssm_backward_chunked(*scan, s["dout"], workspace=wb, **args)
        torch.cuda.synchronize()
    finally:
        lib.mesa_debug_set_wait_limit(-1)
    assert lib.mesa_forward_status_code(ws)[0] == lib.MESA_ERR_TIMEOUT
    assert lib.mesa_forward_status_code(wb)[0] == lib.MESA_ERR_TIMEOUT
    again, S2 = forward(lib, s, workspace=ws)
    assert torch.equal(out, again) and torch.equal(S, S2)
    r = lib.mesa_ssm_backward_chunked(*scan, s["dout"], workspace=wb, **args)
    assert all(torch.equal(x, y) for x, y in zip(grads, r))
    assert lib.mesa_forward_status_code(ws)[0] == lib.MESA_OK and lib.mesa_forward_status_code(wb)[0] == lib.MESA_OK
